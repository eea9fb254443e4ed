"""Cases, plain forms and 64-bit values of the block norms, the grouped products and the AdamW step.

Three sets of operators stand around the MoE layer in a training or serving step:

  block norms       x = RMSNorm(u) w before the layer, and behind it the sum of the expert
                    outputs, its norm, the gate, the residual and the next block's norm in one
                    pass (`moe_norm`, `moe_combine_norm`, and their backward passes)
  grouped products  one weight matrix per expert applied to that expert's rows of a ragged row
                    list (`moe_grouped_mm`), with the gradients of the rows and of the weights
                    (`moe_grouped_mm_dx`, `moe_grouped_mm_dw`)
  AdamW             one step over a list of fp32 master tensors with 32-bit or 8-bit moments
                    (`moe_adamw`)

With `own` false, `run` computes a case with elementary torch operations in 32 bits; with `own`
true it makes the calls a user of the library makes.
"""
import itertools
import math

import torch

own = False

EPS = 1e-6
BETA1, BETA2, ADAM_EPS, LR, DECAY = 0.9, 0.95, 1e-8, 3e-4, 0.1
BLOCK = 128                 # elements that share a scale in the 8-bit states


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one generated token through the end of a block: 8 routed + 1 shared expert rows, the
        # residual and the next block's norm; latency only
        dict(name="combine_token", op="combine", T=1, d=7168, slots=9, gate_group=1 << 20,
             res=1.0, train=False, dtype="bf16"),
        # a long prompt or a training batch through the end of a block, with what the backward needs
        dict(name="combine_batch", op="combine", T=16384, d=7168, slots=9, gate_group=1 << 20,
             res=0.5, train=True, dtype="bf16"),
        # the norm before a small fp32 layer, rows of an odd length
        dict(name="norm_f32_odd", op="norm", T=4097, d=1001, dtype="f32"),
        # backward through the norm before a layer, joined with the residual's gradient
        dict(name="norm_backward", op="norm_backward", T=8192, d=5120, res=1.0, dtype="bf16"),
        # backward through the end of a block whose gate is shared by the tokens of a sequence
        dict(name="combine_backward", op="combine_backward", T=8191, d=2048, gate_group=1024,
             dtype="bf16"),
        # the experts of one generated token: six matrices of 64, one row each
        dict(name="mm_token", op="mm", groups=64, rows=6, d_in=2048, d_out=2816, skew=0.0),
        # ordinary training batch, unevenly loaded experts, rows that start anywhere
        dict(name="mm_batch", op="mm", groups=64, rows=24570, d_in=2048, d_out=2816, skew=0.6),
        # gradient of the rows through wide down projections
        dict(name="mm_dx_batch", op="mm_dx", groups=32, rows=32768, d_in=2048, d_out=7168,
             skew=0.3),
        # weight gradients of ragged groups in bf16
        dict(name="mm_dw_ragged", op="mm_dw", groups=64, rows=24571, d_in=2048, d_out=1408,
             skew=0.6, grads="bf16", accumulate=False),
        # the norm weights, gates and router of a small model: many tensors, some of odd length
        dict(name="adamw_small", op="adamw", tensors=96, numel=20000, bits=32, grads="f32"),
        # one rank's experts with fp32 moments, gradients as the bf16 backward leaves them
        dict(name="adamw_experts", op="adamw", tensors=7, numel=60000001, bits=32, grads="bf16"),
        # the same with 8-bit moments
        dict(name="adamw_experts_8bit", op="adamw", tensors=7, numel=60000001, bits=8,
             grads="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["combine", "norm", "norm_backward", "combine_backward", "mm", "mm_dx",
                     "mm_dw", "mm_dw", "adamw", "adamw"])
    if op in ("combine", "norm", "norm_backward", "combine_backward"):
        dtype = rng.choice(["bf16", "bf16", "f32"])
        d = _log(rng, 64, 7168)
        d = d if rng.random() < 0.3 else max(64, d // 64 * 64)
        case = dict(op=op, T=_log(rng, 1, 16384), d=d, dtype=dtype)
        slots = rng.choice([1, 2, 7, 9])
        if op == "combine":
            most = 16384 * 7168 * 9 // (case["d"] * (slots + 2)) // (2 if dtype == "f32" else 1)
            case["T"] = min(case["T"], most)
            case.update(slots=slots, train=rng.random() < 0.5)
        if op in ("combine", "norm_backward"):
            case["res"] = rng.choice([1.0, 0.5, 2.0])
        if op in ("combine", "combine_backward"):
            case["gate_group"] = rng.choice([0, 1, 1 << 20, _log(rng, 2, 5000)])
        return case
    if op == "adamw":
        tensors = _log(rng, 1, 300)
        return dict(op=op, tensors=tensors, bits=rng.choice([8, 32]),
                    grads=rng.choice(["f32", "bf16"]),
                    numel=_log(rng, 100, min(4e7, 4e8 / tensors)))
    groups = _log(rng, 1, 128)
    case = dict(op=op, groups=groups, rows=_log(rng, 1, 24000), d_in=8 * _log(rng, 8, 512),
                d_out=8 * _log(rng, 8, 512), skew=rng.choice([0.0, 0.3, 0.6]))
    while case["groups"] * case["d_in"] * case["d_out"] > 500e6:
        case["groups"] = max(1, case["groups"] // 2)
    if op == "mm_dw":
        case["grads"] = rng.choice(["f32", "bf16"])
        case["accumulate"] = case["grads"] == "f32" and rng.random() < 0.5
    return case


# ------------------------------------------------------------------------------------ inputs
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _size(case):
    return 2 if case["dtype"] == "bf16" else 4


def _gate_rows(case):
    g = case["gate_group"]
    return (case["T"] + g - 1) // g if g else 0


def _loads(case):
    """Rows of each group: 1 / rank^skew of them, the ranks shuffled, summing to `rows`."""
    G, R = case["groups"], case["rows"]
    order = torch.randperm(G, generator=torch.Generator().manual_seed(G * 131 + R))
    p = (order + 1).double() ** -case["skew"]
    edge = torch.round(torch.cumsum(p, 0) / p.sum() * R).long()
    edge[-1] = R
    return torch.diff(edge, prepend=torch.zeros(1, dtype=torch.long))


def _numels(case):
    """Lengths of the tensor list: around `numel`, most of them not a multiple of anything."""
    n, k = case["numel"], case["tensors"]
    return [max(1, n - (n // 3) * (i % 3) // 2 - (i * 37) % 61 * (i > 0)) for i in range(k)]


def _places(ns):
    """Where each tensor starts in a flat buffer that holds them all, every one from a multiple
    of BLOCK elements on, and the buffer's length."""
    whole = [(n + BLOCK - 1) // BLOCK * BLOCK for n in ns]
    ends = list(itertools.accumulate(whole))
    return [e - w for e, w in zip(ends, whole)], ends[-1]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)

    def normal(*shape, std=1.0, dtype=torch.float32):
        out = torch.empty(shape, dtype=dtype, device="cuda")
        return out.normal_(0.0, std, generator=gen)

    s = dict(case=case)
    op = case["op"]
    if op in ("combine", "norm", "norm_backward", "combine_backward"):
        T, d, dt = case["T"], case["d"], _TYPES[case["dtype"]]
        act = dict(dtype=dt, device="cuda")
        s["w"] = (1.0 + normal(d, std=0.1)).to(dt)
        if op == "norm":
            s.update(x=normal(T, d, std=2.0, dtype=dt), out=torch.empty(T, d, **act))
        elif op == "norm_backward":
            s.update(x=normal(T, d, std=2.0, dtype=dt), dout=normal(T, d, std=0.1, dtype=dt),
                     dh=normal(T, d, std=0.1, dtype=dt), dx=torch.empty(T, d, **act),
                     dw=torch.empty(d, device="cuda"))
        else:
            n_gate = _gate_rows(case)
            s["gate"] = (0.5 + normal(n_gate, d, std=0.2)).to(dt) if n_gate else None
            if op == "combine":
                s.update(u=normal(T, d, std=2.0, dtype=dt),
                         y_slots=normal(T, case["slots"], d, std=0.3, dtype=dt),
                         w_next=(1.0 + normal(d, std=0.1)).to(dt), h=torch.empty(T, d, **act),
                         x_next=torch.empty(T, d, **act),
                         y=torch.empty(T, d, **act) if case["train"] else None)
            else:
                s.update(y=normal(T, d, std=0.7, dtype=dt), dh=normal(T, d, std=0.1, dtype=dt),
                         dy=torch.empty(T, d, **act), dw=torch.empty(d, device="cuda"),
                         dgate=torch.empty(n_gate, d, **act) if n_gate else None)
        if own:
            import forward_moe_route_b200 as moe
            s["desc"] = moe.make_norm_desc(T, d, EPS, case["dtype"], case.get("slots", 1),
                                           case.get("gate_group", 0), case.get("res", 1.0))
            if op in ("norm_backward", "combine_backward"):
                s["ws"] = moe.norm_backward_workspace(s["desc"])
        return s
    if op in ("mm", "mm_dx", "mm_dw"):
        G, R, d_in, d_out = case["groups"], case["rows"], case["d_in"], case["d_out"]
        bf = dict(dtype=torch.bfloat16, device="cuda")
        loads = _loads(case)
        s["loads"] = loads.tolist()
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.long),
                                  torch.cumsum(loads, 0)]).to(torch.int32).cuda()
        if op != "mm_dx":
            s["x"] = normal(R, d_in, dtype=torch.bfloat16)
        if op != "mm":
            s["dy"] = normal(R, d_out, dtype=torch.bfloat16)
        if op != "mm_dw":
            s["w"] = normal(G, d_out, d_in, std=0.02, dtype=torch.bfloat16)
        if op == "mm":
            s["y"] = torch.empty(R, d_out, **bf)
        elif op == "mm_dx":
            s["dx"] = torch.empty(R, d_in, **bf)
        elif case["accumulate"]:
            s["dw"] = normal(G, d_out, d_in)
        else:
            s["dw"] = torch.empty(G, d_out, d_in, dtype=_TYPES[case["grads"]], device="cuda")
        return s
    # the tensors are pieces of flat buffers, as a trainer lays them out; the gaps between them
    # hold zeros
    ns = _numels(case)
    starts, total = _places(ns)
    there = torch.zeros(total, dtype=torch.bool, device="cuda")
    for a, n in zip(starts, ns):
        there[a:a + n] = True
    s.update(step=12, seed=seed, ns=ns, starts=starts)
    s["p"] = normal(total, std=0.02).mul_(there)
    s["grad"] = normal(total, std=1e-3, dtype=_TYPES[case["grads"]]).mul_(there)
    s["p_bf16"] = s["p"].to(torch.bfloat16)
    if case["bits"] == 32:
        s["m"] = normal(total, std=3e-4).mul_(there)
        s["v"] = normal(total, std=6e-4).square_().mul_(there)
    else:
        # codes as earlier steps leave them: signed first moments, roots of the second above zero
        def codes():
            return torch.randint(1, 0x7f, (total,), generator=gen, device="cuda",
                                 dtype=torch.uint8).mul_(there)
        s["m"] = (codes() ^ (codes() << 7)).mul_(there).view(torch.float8_e4m3fn)
        s["v"] = codes().view(torch.float8_e4m3fn)
        s["m_scale"] = normal(total // BLOCK, std=2e-6).abs_()
        s["v_scale"] = normal(total // BLOCK, std=4e-6).abs_().add_(1e-6)
    if own:
        import forward_moe_route_b200 as moe
        at = [slice(a, a + n) for a, n in zip(starts, ns)]
        blocks = [slice(a // BLOCK, -(-(a + n) // BLOCK)) for a, n in zip(starts, ns)]
        lists = {k: [s[k][i] for i in at] for k in ("p", "grad", "m", "v", "p_bf16")}
        scales = {k: [s[k][i] for i in blocks] for k in ("m_scale", "v_scale") if k in s}
        s["desc"] = moe.make_adamw_desc(LR, BETA1, BETA2, ADAM_EPS, case["bits"], seed)
        s["table"] = moe.adamw_table(lists["p"], lists["grad"], lists["m"], lists["v"],
                                     p_bf16=lists["p_bf16"], weight_decay=DECAY, **scales)
    return s


# ------------------------------------------------------------------------------------ plain forms
def _rms(x):
    return torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def _gate_of_rows(case, gate):
    if gate is None:
        return 1.0
    at = torch.arange(case["T"], device="cuda") // case["gate_group"]
    return gate.float()[at] if gate.shape[0] > 1 else gate.float()


def _plain_norm(s):
    x = s["x"].float()
    return (x * _rms(x) * s["w"].float()).to(s["x"].dtype)


def _norm_gradient(x, c):
    """Gradient of x / rms(x) for the gradient c of its result."""
    r = _rms(x)
    n = x * r
    return r * (c - n * (c * n).mean(-1, keepdim=True)), n


def _plain_norm_backward(s):
    x, g = s["x"].float(), s["dout"].float()
    dx, n = _norm_gradient(x, g * s["w"].float())
    dw = (g * n).double().sum(0).float()
    return (s["case"]["res"] * s["dh"].float() + dx).to(s["x"].dtype), dw


def _plain_combine(s):
    case = s["case"]
    y = s["y_slots"].float().sum(1)
    n = y * _rms(y) * s["w"].float()
    h = case["res"] * s["u"].float() + _gate_of_rows(case, s["gate"]) * n
    x = h * _rms(h) * s["w_next"].float()
    dt = s["u"].dtype
    return h.to(dt), x.to(dt), y.to(dt) if case["train"] else None


def _plain_combine_backward(s):
    case = s["case"]
    y, dh, w = s["y"].float(), s["dh"].float(), s["w"].float()
    gate = _gate_of_rows(case, s["gate"])
    dy, n = _norm_gradient(y, dh * gate * w)
    dw = (dh * gate * n).double().sum(0).float()
    dgate = None
    if s["gate"] is not None:
        at = torch.arange(case["T"], device="cuda") // case["gate_group"]
        dgate = torch.zeros(s["gate"].shape, dtype=torch.float64, device="cuda")
        dgate = dgate.index_add_(0, at, (dh * w * n).double()).to(s["y"].dtype)
    return dy.to(s["y"].dtype), dw, dgate


def _groups(s):
    """(group, its rows) of every group that has any."""
    ends = itertools.accumulate(s["loads"])
    return [(g, slice(e - n, e)) for g, (n, e) in enumerate(zip(s["loads"], ends)) if n]


def _plain_mm(s):
    x = s["x"].float()
    return torch.cat([x[r] @ s["w"][g].float().T for g, r in _groups(s)]).to(torch.bfloat16)


def _plain_mm_dx(s):
    dy = s["dy"].float()
    return torch.cat([dy[r] @ s["w"][g].float() for g, r in _groups(s)]).to(torch.bfloat16)


def _plain_mm_dw(s):
    dy, x, dw = s["dy"].float(), s["x"].float(), s["dw"]
    if not s["case"]["accumulate"]:
        dw.zero_()
    [dw[g].add_(dy[r].T @ x[r]) if s["case"]["accumulate"] else dw[g].copy_(dy[r].T @ x[r])
     for g, r in _groups(s)]
    return dw


_LOW = 0xffffffff


def _random_words(s):
    """32 random bits per element: Philox-2x32 with 7 rounds (Salmon et al., "Parallel random
    numbers: as easy as 1, 2, 3", SC 2011) of the pair's index in its tensor and the tensor's
    place in the list, keyed by seed and step; an element takes the word of its parity."""
    ends = s["starts"][1:] + [len(s["p"])]
    whole = torch.tensor([e - a for a, e in zip(s["starts"], ends)], device="cuda")
    t = torch.repeat_interleave(torch.arange(len(whole), device="cuda"), whole)
    i = torch.arange(len(t), device="cuda") - torch.tensor(s["starts"], device="cuda")[t]
    j = i >> 1
    a, b = j & _LOW, ((t << 8) ^ (j >> 32)) & _LOW
    key = ((s["seed"] ^ (s["seed"] >> 32)) + s["step"] * 0x9E3779B9) & _LOW
    for _ in range(7):
        p = a * 0xD256D193
        a, b = ((p >> 32) & _LOW) ^ key ^ b, p & _LOW
        key = (key + 0x9E3779B9) & _LOW
    return torch.where(i % 2 == 1, b, a)


def _encode(x, bits16):
    """E4M3 codes of x, |x| <= 448, rounded up with the probability of its distance."""
    a = x.abs()
    word = a.view(torch.int32).long() + (bits16 << 4)
    normal = (word >> 20) - 960
    small = torch.floor(a * 512.0 + bits16.float() * 2.0 ** -16).long()
    c = torch.where(a >= 2.0 ** -6, normal, small).clamp_(max=0x7e)
    return c + 128 * (x < 0)


def _scaled(x):
    """The scale of each block and the block's values over it."""
    x = x.view(-1, BLOCK)
    most = x.abs().amax(1, keepdim=True)
    there = most >= 2.0 ** -100
    one = torch.ones_like(most)
    scale = torch.where(there, most / 448.0, 0 * one)
    inverse = torch.where(there, 448.0 / torch.where(there, most, one), 0 * one)
    return scale[:, 0], (x * inverse).view(-1)


def _plain_adamw(s):
    f = lambda v: torch.tensor(v, dtype=torch.float32, device="cuda")  # noqa: E731
    g, p, m, v = s["grad"].float(), s["p"], s["m"].float(), s["v"].float()
    small = s["case"]["bits"] == 8
    if small:
        m = (m.view(-1, BLOCK) * s["m_scale"][:, None]).view(-1)
        v = (v.view(-1, BLOCK) * s["v_scale"][:, None]).view(-1).square()
    m = f(BETA1) * m + f(1 - BETA1) * g
    v = f(BETA2) * v + f(1 - BETA2) * (g * g)
    root = v.sqrt()
    down = root * f(1 / math.sqrt(1 - BETA2 ** s["step"])) + f(ADAM_EPS)
    p.copy_(p * f(1 - LR * DECAY) - m * f(LR / (1 - BETA1 ** s["step"])) / down)
    s["p_bf16"].copy_(p)
    if not small:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return _adamw_outputs(s)
    word = _random_words(s)
    scale, x = _scaled(m)
    s["m_scale"].copy_(scale)
    s["m"].view(torch.uint8).copy_(_encode(x, word & 0xffff))
    scale, x = _scaled(root)
    s["v_scale"].copy_(scale)
    code = _encode(x, word >> 16)
    s["v"].view(torch.uint8).copy_(torch.where((code == 0) & (root > 0), 1, code))
    return _adamw_outputs(s)


def _adamw_outputs(s):
    """The updated state, in the flat buffers that hold it."""
    return {k: s[k] for k in ("p", "p_bf16", "m", "v", "m_scale", "v_scale") if k in s}


# ------------------------------------------------------------------------------------ one pass
def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"norm": _plain_norm, "norm_backward": _plain_norm_backward,
                "combine": _plain_combine, "combine_backward": _plain_combine_backward,
                "mm": _plain_mm, "mm_dx": _plain_mm_dx, "mm_dw": _plain_mm_dw,
                "adamw": _plain_adamw}[op](s)
    import forward_moe_route_b200 as moe
    if op == "norm":
        moe.moe_norm(s["desc"], s["x"], s["w"], s["out"])
        return s["out"]
    if op == "norm_backward":
        moe.moe_norm_backward(s["desc"], s["x"], s["w"], s["dout"], s["dh"], s["dx"], s["dw"],
                              s["ws"])
        return s["dx"], s["dw"]
    if op == "combine":
        moe.moe_combine_norm(s["desc"], s["u"], s["y_slots"], s["w"], s["gate"], s["w_next"],
                             s["h"], s["y"], s["x_next"])
        return s["h"], s["x_next"], s["y"]
    if op == "combine_backward":
        moe.moe_combine_norm_backward(s["desc"], s["y"], s["w"], s["gate"], s["dh"], s["dy"],
                                      s["dw"], s["dgate"], s["ws"])
        return s["dy"], s["dw"], s["dgate"]
    if op == "mm":
        moe.moe_grouped_mm(s["x"], s["w"], s["offsets"], s["y"])
        return s["y"]
    if op == "mm_dx":
        moe.moe_grouped_mm_dx(s["dy"], s["w"], s["offsets"], s["dx"])
        return s["dx"]
    if op == "mm_dw":
        moe.moe_grouped_mm_dw(s["dy"], s["x"], s["offsets"], s["dw"],
                              accumulate=s["case"]["accumulate"])
        return s["dw"]
    moe.moe_adamw(s["desc"], s["table"], s["step"])
    return _adamw_outputs(s)


# ------------------------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    if op in ("combine", "norm", "norm_backward", "combine_backward"):
        T, d, b = case["T"], case["d"], _size(case)
        if op == "norm":
            return dict(bytes=(2 * T + 1) * d * b, flops=5.0 * T * d)
        if op == "norm_backward":
            return dict(bytes=(4 * T + 1) * d * b + 4 * d, flops=12.0 * T * d)
        if op == "combine":
            rows = T * (case["slots"] + 3 + bool(case["train"])) + _gate_rows(case) + 2
            return dict(bytes=rows * d * b, flops=(case["slots"] + 12.0) * T * d)
        return dict(bytes=(3 * T + 2 * _gate_rows(case) + 1) * d * b + 4 * d, flops=16.0 * T * d)
    if op in ("mm", "mm_dx", "mm_dw"):
        R, d_in, d_out = case["rows"], case["d_in"], case["d_out"]
        used = int((_loads(case) > 0).sum())
        moved = 2.0 * R * (d_in + d_out)
        if op != "mm_dw":
            moved += 2.0 * used * d_in * d_out
        elif case["accumulate"]:
            moved += 8.0 * used * d_in * d_out
        else:
            moved += (2.0 if case["grads"] == "bf16" else 4.0) * case["groups"] * d_in * d_out
        return dict(bytes=moved, flops=2.0 * R * d_in * d_out)
    n = float(sum(_numels(case)))
    each = 8 + 2 + (2 if case["grads"] == "bf16" else 4)
    each += 16 if case["bits"] == 32 else 4 + 16.0 / BLOCK
    return dict(bytes=n * each, flops=15.0 * n)


# ------------------------------------------------------------------------------------ 64 bits
def _exact_normed(x):
    return x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()


def _exact_norm_gradient(x, c):
    """With q = mean(x^2) + eps: d/dx (x q^-1/2) . c = q^-1/2 c - q^-3/2 x <x, c> / d."""
    q = x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS
    return c * q.pow(-0.5) - x * q.pow(-1.5) * ((x * c).sum(-1, keepdim=True) / x.shape[-1])


def exact(case, seed):
    keep, globals()["own"] = own, False
    try:
        s = prepare(case, seed)
    finally:
        globals()["own"] = keep
    op, D = case["op"], torch.float64
    if op == "norm":
        return _exact_normed(s["x"].to(D)) * s["w"].to(D)
    if op == "norm_backward":
        x, g, w = s["x"].to(D), s["dout"].to(D), s["w"].to(D)
        return (_exact_norm_gradient(x, g * w) + s["dh"].to(D) * case["res"],
                (_exact_normed(x) * g).sum(0))
    if op in ("combine", "combine_backward"):
        T, w = case["T"], s["w"].to(D)
        if s["gate"] is None:
            gate = torch.ones(T, 1, dtype=D, device="cuda")
        else:
            gate = s["gate"].to(D).repeat_interleave(min(case["gate_group"], T), 0)[:T]
        if op == "combine":
            y = torch.zeros(T, case["d"], dtype=D, device="cuda")
            for k in range(case["slots"]):
                y += s["y_slots"][:, k].to(D)
            h = s["u"].to(D).mul_(case["res"]).addcmul_(gate, _exact_normed(y) * w)
            return h, _exact_normed(h) * s["w_next"].to(D), y if case["train"] else None
        y, dh = s["y"].to(D), s["dh"].to(D)
        n = _exact_normed(y)
        dgate = None
        if s["gate"] is not None:
            # sums over each run of gate_group rows, the last one padded with zeros
            run_rows = min(case["gate_group"], T)
            t = dh * n * w
            t = torch.cat([t, t.new_zeros(-T % run_rows, case["d"])])
            dgate = t.view(-1, run_rows, case["d"]).sum(1)
        return _exact_norm_gradient(y, dh * w * gate), (dh * gate * n).sum(0), dgate
    if op in ("mm", "mm_dx", "mm_dw"):
        at, parts = 0, []
        for g, n in enumerate(s["loads"]):
            rows = slice(at, at + n)
            at += n
            if op == "mm":
                parts.append(s["x"][rows].to(D) @ s["w"][g].to(D).T)
            elif op == "mm_dx":
                parts.append(s["dy"][rows].to(D) @ s["w"][g].to(D))
            else:
                t = s["dy"][rows].to(D).T @ s["x"][rows].to(D)
                parts.append(t + s["dw"][g].to(D) if case["accumulate"] else t)
        return torch.stack(parts) if op == "mm_dw" else torch.cat(parts)
    # AdamW: the update from the moments as they are held.  The new 8-bit codes are drawn at
    # random between two neighbours, so they have no value here; their scales have.
    t, g, p, m, v = s["step"], s["grad"].to(D), s["p"].to(D), s["m"].to(D), s["v"].to(D)
    if case["bits"] == 8:
        m *= s["m_scale"].to(D).repeat_interleave(BLOCK)
        v = (v * s["v_scale"].to(D).repeat_interleave(BLOCK)) ** 2
    m = m + (1 - BETA1) * (g - m)
    v = v + (1 - BETA2) * (g * g - v)
    p = p - LR * (DECAY * p + (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt() + ADAM_EPS))
    if case["bits"] == 32:
        return dict(p=p, p_bf16=p, m=m, v=v)
    return dict(p=p, p_bf16=p, m=None, v=None,
                m_scale=m.abs().view(-1, BLOCK).max(1).values / 448,
                v_scale=v.view(-1, BLOCK).max(1).values.sqrt() / 448)
