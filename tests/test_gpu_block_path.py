"""A block from the framework's own layer and the operators around it, as a trainer runs them: norm,
routing, permutation, experts, the end of the block from the experts' rows, and in reverse the two
norms, the layer's backward on the gradient of the sum, and the AdamW step on its bf16 gradients.

The gradients are held against fp64 differentiation of the same block (torch autograd of the
formulas, the choice of experts taken from the routing).  Tolerance, relative in the Frobenius norm:
between u and any gradient there are at most 14 roundings to bf16 (x, a, b, the experts' rows, their
weighted outputs, y, h, x_next; dh, dy, the experts' dz, da, db, dx and the gradient itself),
each at most 2^-8 of what it rounds, and each may add that much to the end: 14 2^-8 = 5.5%.  A
gradient that went the wrong way or twice is off by tens of percent.

The router's gradient comes from dg_k = <dy, z_k>, and no rounding of dy or of an expert's output
z_k is relative to that product: it moves dg_k by up to 2^-8 b_k, b_k = |dy| |z_k|, which at 256
columns is about 16 times a typical <dy, z_k>.  With S the sum of the chosen affinities s_k the gate
weights' gradient is ds_k = (dg_k - sum_j dg_j s_j / S) / S, so it moves by up to
2^-8 (b_k + sum_j b_j s_j / S) / S, dl_k = ds_k s_k (1 - s_k) by s_k (1 - s_k) of that, and
dW_r = sum_t dl_t x_t^T by |x_t| times the norm of that over k, for each token.  Over hundreds of
tokens these errors have either sign and 5.5% of the whole holds; a single token is held to 14 times
that size.
"""
import pytest
import torch

import forward_moe_route_b200 as moe

pytestmark = pytest.mark.gpu

D, INNER, N, K, KS = 256, 128, 8, 2, 1
EPS, RES, SCALE = 1e-5, 0.5, 1.0
BF = dict(dtype=torch.bfloat16, device="cuda")
I32 = dict(dtype=torch.int32, device="cuda")


class Block:
    def __init__(self, T, group, seed=1):
        gen = torch.Generator().manual_seed(seed)
        self.T, self.group = T, group
        S, R, E = K + KS, T * K, N + KS

        def draw(*shape, std=1.0, mean=0.0):
            return (torch.randn(*shape, generator=gen) * std + mean).to(torch.bfloat16).cuda()

        self.w = dict(w1=draw(D, std=0.1, mean=1.0), w2=draw(D, std=0.1, mean=1.0),
                      w3=draw(D, std=0.1, mean=1.0), gate=draw(-(-T // group), D, std=0.1, mean=0.5),
                      router=draw(N, D, std=0.06), gu=draw(E, 2 * INNER, D, std=0.06),
                      down=draw(E, D, INNER, std=0.08))
        self.g = {k: torch.full_like(v, float("nan")) for k, v in self.w.items()}
        for k in ("w1", "w2", "w3"):
            self.g[k] = torch.full((D,), float("nan"), device="cuda")
        self.u, self.g_next, self.g_h = draw(T, D), draw(T, D), draw(T, D)
        self.layer = moe.make_desc(T, D, KS, N, K, INNER, "sigmoid", True, SCALE)
        self.norm = moe.make_norm_desc(T, D, EPS, res_scale=RES)
        self.next = moe.make_norm_desc(T, D, EPS)
        self.end = moe.make_norm_desc(T, D, EPS, n_slots=S, gate_group=group, res_scale=RES)
        self.ws, self.back_ws = moe.workspace(self.layer), moe.backward_workspace(self.layer)
        self.norm_ws = moe.norm_backward_workspace(self.norm)
        self.end_ws = moe.norm_backward_workspace(self.end)
        rows = {k: torch.empty(T, D, **BF) for k in ("x", "h", "y", "x_next", "dh", "dy", "dx", "du")}
        self.b = dict(rows, slots=torch.empty(T, S, D, **BF), x_perm=torch.empty(R, D, **BF),
                      idx=torch.empty(T, K, **I32), weight=torch.empty(T, K, device="cuda"),
                      counts=torch.empty(N, **I32), offsets=torch.empty(N + 1, **I32),
                      src=torch.empty(R, **I32), slot=torch.empty(R, **I32))
        self.master = {k: v.float() for k, v in self.w.items()}
        zeros = [[torch.zeros(v.numel(), device="cuda") for v in self.w.values()] for _ in range(2)]
        names = list(self.w)
        self.adam = moe.make_adamw_desc(1e-3)
        self.table = moe.adamw_table([self.master[k] for k in names], [self.g[k] for k in names],
                                     *zeros, p_bf16=[self.w[k] for k in names], weight_decay=0.1)
        self.step_no = torch.zeros(1, **I32)

    def gradients(self):
        b, w, g = self.b, self.w, self.g
        moe.moe_norm(self.norm, self.u, w["w1"], b["x"])
        moe.moe_route(self.layer, b["x"], w["router"], None, b["idx"], b["weight"], b["counts"],
                      self.ws)
        moe.moe_permute(self.layer, b["x"], b["idx"], b["counts"], b["offsets"], b["src"],
                        b["slot"], b["x_perm"], None, self.ws)
        moe.moe_grouped_swiglu(self.layer, b["x"], b["x_perm"], None, b["offsets"], b["src"],
                               b["slot"], b["weight"], w["gu"], None, w["down"], None, b["slots"],
                               self.ws)
        moe.moe_combine_norm(self.end, self.u, b["slots"], w["w2"], w["gate"], w["w3"], b["h"],
                             b["y"], b["x_next"])
        moe.moe_norm_backward(self.next, b["h"], w["w3"], self.g_next, self.g_h, b["dh"], g["w3"],
                              self.norm_ws)
        moe.moe_combine_norm_backward(self.end, b["y"], w["w2"], w["gate"], b["dh"], b["dy"],
                                      g["w2"], g["gate"], self.end_ws)
        moe.moe_backward_bf16_grads(self.layer, b["x"], w["router"], None, w["gu"], w["down"],
                                    b["dy"], b["dx"], g["router"], g["gu"], g["down"],
                                    self.back_ws)
        moe.moe_norm_backward(self.norm, self.u, w["w1"], b["dx"], b["dh"], b["du"], g["w1"],
                              self.norm_ws)

    def step(self):
        self.step_no += 1
        self.gradients()
        moe.moe_adamw(self.adam, self.table, self.step_no)

    def tensors(self):
        return (list(self.w.values()) + list(self.master.values()) + list(self.g.values()) +
                [self.b["x_next"], self.b["du"]])


def exact(m):
    """(h, x_next, gradients) of the block in fp64, and the size that an error of the router's
    gradient is relative to, over 2^-8 a rounding (above)."""
    leaf = {k: v.double().requires_grad_() for k, v in m.w.items()}
    leaf["u"] = m.u.double().requires_grad_()
    idx = m.b["idx"].long()

    def norm(v):
        return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)

    x = norm(leaf["u"]) * leaf["w1"]
    s = torch.sigmoid(x @ leaf["router"].T).gather(1, idx)
    weight = SCALE * s / s.sum(1, keepdim=True)

    def expert(e, rows):
        a, b = (rows @ leaf["gu"][e].T).split(INNER, 1)
        return (torch.nn.functional.silu(a) * b) @ leaf["down"][e].T

    y = sum(expert(e, x) for e in range(KS))
    z = torch.zeros(m.T, K, dtype=torch.float64, device="cuda")
    for e in range(N):
        t, k = (idx == e).nonzero(as_tuple=True)
        out = expert(KS + e, x[t])
        z[t, k] = out.detach().norm(dim=1)
        y = y.index_add(0, t, out * weight[t, k][:, None])
    y.retain_grad()
    rows = torch.arange(m.T, device="cuda") // m.group
    h = RES * leaf["u"] + leaf["gate"][rows] * norm(y) * leaf["w2"]
    x_next = norm(h) * leaf["w3"]
    loss = (x_next * m.g_next.double()).sum() + (h * m.g_h.double()).sum()
    loss.backward()
    s, total = s.detach(), s.detach().sum(1, keepdim=True)
    b = y.grad.norm(dim=1, keepdim=True) * z
    dl = SCALE / total * (b + (b * s).sum(1, keepdim=True) / total) * s * (1 - s)
    size = float((dl.norm(dim=1) * x.detach().norm(dim=1)).sum())
    return h.detach(), x_next.detach(), {k: v.grad for k, v in leaf.items()}, size


@pytest.mark.parametrize("T,group", [(333, 100), (333, 1), (333, 1 << 20), (1, 1), (1500, 3)])
def test_gradients_of_a_block(T, group):
    m = Block(T, group)
    m.gradients()
    assert moe.moe_last_device_status() == moe.OK
    h, x_next, want, router = exact(m)
    got = dict(m.g, u=m.b["du"], h=m.b["h"], x_next=m.b["x_next"])
    want.update(h=h, x_next=x_next)
    for k, w in want.items():
        g = got[k].double()
        assert g.shape == w.shape and g.isfinite().all(), k
        size = router if k == "router" and T == 1 else float(w.norm())
        off = float((g - w).norm())
        assert off <= 14 * 2.0 ** -8 * size, f"{k}: {off / size:.4f}"


def test_captured_steps_repeat_eager_ones():
    eager, held = Block(333, 100), Block(333, 100)
    for m in (eager, held):
        m.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held.step()
    for _ in range(3):
        graph.replay()
        eager.step()
    assert int(held.step_no) == int(eager.step_no) == 4
    for a, b in zip(eager.tensors(), held.tensors()):
        assert a.float().isfinite().all() and torch.equal(a, b)
    assert moe.moe_last_device_status() == moe.OK
