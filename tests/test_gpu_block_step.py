"""One training step of a block from the operators around the layer, as a trainer runs them: the
norm, routing, linear experts as grouped products, the end of the block, the same in reverse, and
the AdamW step over every weight, which writes the bf16 copies that the next step reads.

Each operator's output is held against the fp64 oracle on the inputs it really had, within the
tolerances of that operator's own tests; then the whole step is captured into a graph, and its
replay must leave the same bits as the same steps run eagerly.
"""
import numpy as np
import pytest
import torch

import forward_moe_route_b200 as moe
from oracle import block
from test_gpu_block_norm import close as norm_close, f64, sums_close
from test_gpu_grouped import close as product_close

pytestmark = pytest.mark.gpu

T, D, INNER, N, K = 333, 256, 136, 8, 2
EPS, RES, GROUP = 1e-5, 0.5, 100
BF = dict(dtype=torch.bfloat16, device="cuda")


class Block:
    """The block's weights, buffers and step."""

    def __init__(self, bits, seed=1):
        gen = torch.Generator().manual_seed(seed)

        def draw(*shape, std=1.0, mean=0.0):
            return (torch.randn(*shape, generator=gen) * std + mean).cuda()

        master = {"w1": draw(D, std=0.1, mean=1.0), "w2": draw(D, std=0.1, mean=1.0),
                  "w3": draw(D, std=0.1, mean=1.0), "up": draw(N, INNER, D, std=0.06),
                  "down": draw(N, D, INNER, std=0.08),
                  "gate": draw(-(-T // GROUP), D, std=0.1, mean=0.5)}
        self.w = {k: x.to(torch.bfloat16) for k, x in master.items()}
        self.grad = {k: torch.zeros_like(x) if x.dim() > 1 else
                     torch.zeros(D, device="cuda") for k, x in self.w.items()}
        self.master = master
        self.router = draw(N, D, std=0.3).to(torch.bfloat16)
        self.u, self.g_next, self.g_h = (draw(T, D).to(torch.bfloat16) for _ in range(3))
        names = list(master)
        size = {k: master[k].numel() for k in names}
        if bits == 32:
            state = [[torch.zeros(size[k], device="cuda") for k in names] for _ in range(2)]
            scales = {}
        else:
            state = [[torch.zeros(size[k], dtype=torch.uint8, device="cuda") for k in names]
                     for _ in range(2)]
            scales = {s: [torch.zeros(-(-size[k] // 128), device="cuda") for k in names]
                      for s in ("m_scale", "v_scale")}
        self.state = state[0] + state[1] + [x for v in scales.values() for x in v]
        self.table = moe.adamw_table([master[k] for k in names], [self.grad[k] for k in names],
                                     *state, p_bf16=[self.w[k] for k in names],
                                     weight_decay=[0.1 if k in ("up", "down") else 0.0
                                                   for k in names], **scales)
        self.adam = moe.make_adamw_desc(1e-2, state_bits=bits, seed=5)
        self.layer = moe.make_desc(T, D, 0, N, K, 128, "sigmoid", True, 1.0)
        self.ws = moe.workspace(self.layer)
        self.norm = moe.make_norm_desc(T, D, EPS, res_scale=RES)
        self.plain = moe.make_norm_desc(T, D, EPS)
        self.end = moe.make_norm_desc(T, D, EPS, n_slots=K, gate_group=GROUP, res_scale=RES)
        self.norm_ws = moe.norm_backward_workspace(self.norm)
        self.end_ws = moe.norm_backward_workspace(self.end)
        i32 = dict(dtype=torch.int32, device="cuda")
        R = T * K
        rows = dict(x=D, h=D, y=D, x_next=D, dh=D, dy=D, du=D)
        self.b = {k: torch.empty(T, n, **BF) for k, n in rows.items()}
        self.b.update(a=torch.empty(R, INNER, **BF), out=torch.empty(R, D, **BF),
                      da=torch.empty(R, INNER, **BF), dx_perm=torch.empty(R, D, **BF),
                      x_perm=torch.empty(R, D, **BF), idx=torch.empty(T, K, **i32),
                      weight=torch.empty(T, K, device="cuda"), counts=torch.empty(N, **i32),
                      offsets=torch.empty(N + 1, **i32), src=torch.empty(R, **i32),
                      slot=torch.empty(R, **i32))
        self.step_no = torch.zeros(1, **i32)

    def forward(self):
        b, w = self.b, self.w
        moe.moe_norm(self.norm, self.u, w["w1"], b["x"])
        moe.moe_route(self.layer, b["x"], self.router, None, b["idx"], b["weight"], b["counts"],
                      self.ws)
        moe.moe_permute(self.layer, b["x"], b["idx"], b["counts"], b["offsets"], b["src"],
                        b["slot"], b["x_perm"], None, self.ws)
        moe.moe_grouped_mm(b["x_perm"], w["up"], b["offsets"], b["a"])
        moe.moe_grouped_mm(b["a"], w["down"], b["offsets"], b["out"])
        picked = b["out"][b["slot"].long()].float().view(T, K, D)
        b["slots"] = (picked * b["weight"][..., None]).to(torch.bfloat16)
        moe.moe_combine_norm(self.end, self.u, b["slots"], w["w2"], w["gate"], w["w3"], b["h"],
                             b["y"], b["x_next"])

    def backward(self):
        b, w, g = self.b, self.w, self.grad
        moe.moe_norm_backward(self.plain, b["h"], w["w3"], self.g_next, self.g_h, b["dh"],
                              g["w3"], self.norm_ws)
        moe.moe_combine_norm_backward(self.end, b["y"], w["w2"], w["gate"], b["dh"], b["dy"],
                                      g["w2"], g["gate"], self.end_ws)
        d_slots = (b["dy"].float()[:, None] * b["weight"][..., None]).to(torch.bfloat16)
        b["d_out"] = torch.empty_like(b["out"])
        b["d_out"][b["slot"].long()] = d_slots.view(T * K, D)
        moe.moe_grouped_mm_dx(b["d_out"], w["down"], b["offsets"], b["da"])
        moe.moe_grouped_mm_dw(b["d_out"], b["a"], b["offsets"], g["down"])
        moe.moe_grouped_mm_dx(b["da"], w["up"], b["offsets"], b["dx_perm"])
        moe.moe_grouped_mm_dw(b["da"], b["x_perm"], b["offsets"], g["up"])
        b["dx"] = b["dx_perm"][b["slot"].long()].float().view(T, K, D).sum(1).to(torch.bfloat16)
        moe.moe_norm_backward(self.norm, self.u, w["w1"], b["dx"], b["dh"], b["du"], g["w1"],
                              self.norm_ws)

    def step(self):
        self.step_no += 1
        self.forward()
        self.backward()
        moe.moe_adamw(self.adam, self.table, self.step_no)

    def tensors(self):
        return (list(self.master.values()) + list(self.w.values()) + list(self.grad.values()) +
                self.state + [self.b["x_next"], self.b["du"]])


def test_every_operator_of_a_step_against_the_oracle():
    m = Block(32)
    m.step_no += 1
    w = {k: f64(x) for k, x in m.w.items()}
    m.forward()
    m.backward()
    b = {k: f64(x) if x.is_floating_point() else x.cpu().numpy() for k, x in m.b.items()}
    eps = m.norm.eps
    u = f64(m.u)
    want = block.norm(u, w["w1"], eps)
    norm_close("x", m.b["x"], want, np.abs(want), "bf16")
    off = b["offsets"]
    assert off[-1] == T * K and len(np.unique(b["slot"])) == T * K
    for name, got, x, weight, k in (("a", "a", b["x_perm"], w["up"], D),
                                    ("out", "out", b["a"], w["down"], INNER)):
        zero = np.zeros(b[got].shape)
        product_close(name, m.b[got], block.grouped_mm(x, weight, off, zero),
                      block.grouped_mm(abs(x), abs(weight), off, zero), k)
    h, y, x_next = block.combine_norm(u, b["slots"], w["w2"], w["gate"], GROUP, RES, w["w3"], eps)
    y_mag = np.abs(b["slots"]).sum(1)
    gate = block.gate_rows(w["gate"], GROUP, T)
    h_mag = np.abs(RES * u) + np.abs(gate * w["w2"]) * y_mag * block.inv_rms(y, eps)
    norm_close("y", m.b["y"], y, y_mag, "bf16")
    norm_close("h", m.b["h"], h, h_mag, "bf16")
    norm_close("x_next", m.b["x_next"], x_next,
               np.abs(w["w3"]) * block.inv_rms(h, eps) * (h_mag + np.abs(h)), "bf16")

    def through(name, got, dw, x, weight, up, add, scale):
        want, want_w = block.norm_backward(x, weight, up, add, scale, eps)
        r = block.inv_rms(x, eps)
        c = np.abs(up * weight)
        mag = r * c + np.abs(x) * r ** 3 * np.mean(np.abs(x) * c, -1, keepdims=True)
        norm_close(name, got, want, mag + np.abs(scale * add), "bf16")
        sums_close("dw of " + name, dw, want_w, np.sum(np.abs(up * x * r), 0), T)

    through("dh", m.b["dh"], m.grad["w3"], b["h"], w["w3"], f64(m.g_next), f64(m.g_h), 1.0)
    through("du", m.b["du"], m.grad["w1"], u, w["w1"], b["dx"], b["dh"], RES)
    dy, dw2, dgate = block.combine_norm_backward(b["y"], w["w2"], w["gate"], GROUP, b["dh"], eps)
    r = block.inv_rms(b["y"], eps)
    c = np.abs(b["dh"] * gate * w["w2"])
    norm_close("dy", m.b["dy"], dy, r * c + np.abs(b["y"]) * r ** 3 *
               np.mean(np.abs(b["y"]) * c, -1, keepdims=True), "bf16")
    sums_close("dw2", m.grad["w2"], dw2, np.sum(np.abs(b["dh"] * gate * b["y"] * r), 0), T)
    mag = np.zeros_like(dgate)
    np.add.at(mag, np.arange(T) // GROUP, np.abs(b["dh"] * w["w2"] * b["y"] * r))
    sums_close("dgate", m.grad["gate"], dgate, mag, T, "bf16")
    rows = np.diff(off).reshape(N, 1, 1)
    for name, up, x in (("down", b["d_out"], b["a"]), ("up", b["da"], b["x_perm"])):
        zero = np.zeros(w[name].shape)
        product_close("d" + name, m.grad[name], block.grouped_mm_dw(up, x, off, zero),
                      block.grouped_mm_dw(abs(up), abs(x), off, zero), rows)
    for name, up, weight, k in (("da", b["d_out"], "down", D), ("dx_perm", b["da"], "up", INNER)):
        zero = np.zeros(b[name].shape)
        product_close(name, m.b[name], block.grouped_mm_dx(up, w[weight], off, zero),
                      block.grouped_mm_dx(abs(up), abs(w[weight]), off, zero), k)
    before = {k: f64(x) for k, x in m.master.items()}
    moe.moe_adamw(m.adam, m.table, m.step_no)
    for k, x in m.master.items():
        # from zero moments the first step moves every element by lr, against its gradient's sign,
        # or nearly so where the gradient is next to eps
        g = f64(m.grad[k])
        decay = float(np.float32(0.1)) if k in ("up", "down") else 0.0
        want, _, _ = block.adamw(before[k], g, 0 * g, 0 * g, 1, 1e-2, 0.9, 0.95, 1e-8, decay)
        assert np.abs(f64(x) - want).max() <= 2.0 ** -24 * (24 * 1e-2 + 2 * np.abs(want).max() +
                                                             2 * np.abs(before[k]).max())
        assert torch.equal(m.w[k], x.to(torch.bfloat16))
    assert moe.moe_last_device_status() == moe.OK


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps_repeat_eager_ones(bits):
    eager, held = Block(bits), Block(bits)
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
        assert a.float().isfinite().all() if a.is_floating_point() else True
        assert torch.equal(a, b)
    assert moe.moe_last_device_status() == moe.OK


def test_two_blocks_on_two_streams():
    alone = [Block(32, seed=3), Block(8, seed=4)]
    for m in alone:
        for _ in range(4):
            m.step()
    torch.cuda.synchronize()
    both = [Block(32, seed=3), Block(8, seed=4)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in both]
    for _ in range(4):
        for m, s in zip(both, streams):
            with torch.cuda.stream(s):
                m.step()
    torch.cuda.synchronize()
    for m, n in zip(alone, both):
        for a, b in zip(m.tensors(), n.tensors()):
            assert torch.equal(a, b)
    assert moe.moe_last_device_status() == moe.OK
