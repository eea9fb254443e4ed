"""GPU parity of the norms around the layer (moe_norm, moe_combine_norm and
their backward passes) with the fp64 oracle.

Tolerances, from the arithmetic.  A bf16 output is rounded once: at most 2^-8
of its value.  What it is rounded from is fp32: a row's sum of d terms joined
in a tree has a relative error of a few 2^-24 (all terms of a sum of squares are
positive), and every other step adds 2^-24, so 2^-19 relative to the largest
term covers it.  An output that is a difference of terms (dx, h) is held to that
fraction of the sum of the terms' magnitudes.  Column sums over T tokens run in
up to ceil(T / 592) + 592 / 32 + 32 sequential fp32 additions and the T
products carry a few 2^-24 each: 2^-24 (T / 592 + 80) of the sum of magnitudes.
"""
import numpy as np
import pytest
import torch

import forward_moe_route_b200 as moe
from oracle import block

pytestmark = pytest.mark.gpu

EPS = 1e-5
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
F32 = 2.0 ** -19                       # accumulated fp32 arithmetic, see above


def step(dtype):
    return 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24


def rand(gen, *shape, std=1.0, mean=0.0, dtype="bf16"):
    x = torch.randn(*shape, generator=gen, dtype=torch.float64) * std + mean
    return x.to(TYPES[dtype]).cuda()


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def close(name, got, want, scale, dtype):
    """|got - want| <= rounding of want + F32 * scale, element by element."""
    got = f64(got)
    assert got.shape == want.shape
    off = np.abs(got - want) - step(dtype) * np.abs(want) - F32 * scale
    assert np.isfinite(got).all(), name
    assert (off <= 1e-30).all(), f"{name}: over by {off.max():.3e} at {np.argmax(off)}"


def sums_close(name, got, want, magnitude, T, dtype="f32"):
    got = f64(got)
    tol = 2.0 ** -24 * (T / 592 + 80) * magnitude + step(dtype) * np.abs(want)
    off = np.abs(got - want) - tol
    assert (off <= 1e-30).all(), f"{name}: over by {off.max():.3e}"


# one warp a row (1, 2, 4 vectors a lane), one block a row, single elements,
# rows longer than a block's registers
D = [1, 8, 40, 256, 264, 512, 1000, 1024, 1001, 2048, 5120, 7168, 8200, 9001, 34000]
GATES = [0, 1, 3, 64, 1 << 20]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", D)
def test_norm_and_backward(d, dtype):
    gen = torch.Generator().manual_seed(d)
    for T, res in ((1, 1.0), (37, -0.5), (1301 if d < 6000 else 611, 2.0)):
        x, dout, dh = (rand(gen, T, d, std=s, dtype=dtype) for s in (2.0, 1.0, 1.0))
        w = rand(gen, d, mean=1.0, std=0.2, dtype=dtype)
        desc = moe.make_norm_desc(T, d, EPS, dtype, res_scale=res)
        out = torch.full_like(x, float("nan"))
        moe.moe_norm(desc, x, w, out)
        want = block.norm(f64(x), f64(w), desc.eps)
        close("out", out, want, np.abs(want), dtype)

        for with_dh in (dh, None):
            dx = torch.full_like(x, float("nan"))
            dw = torch.full((d,), float("nan"), device="cuda")
            ws = moe.norm_backward_workspace(desc).fill_(0xff)
            moe.moe_norm_backward(desc, x, w, dout, with_dh, dx, dw, ws)
            want, want_w = block.norm_backward(f64(x), f64(w), f64(dout), f64(with_dh), res,
                                               desc.eps)
            r = block.inv_rms(f64(x), desc.eps)
            c = np.abs(f64(dout) * f64(w))
            scale = r * c + np.abs(f64(x)) * r ** 3 * np.mean(np.abs(f64(x)) * c, -1,
                                                              keepdims=True)
            if with_dh is not None:
                scale = scale + np.abs(res * f64(dh))
            close("dx", dx, want, scale, dtype)
            sums_close("dw", dw, want_w, np.sum(np.abs(f64(dout) * f64(x) * r), 0), T)
    assert moe.moe_last_device_status() == moe.OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [8, 264, 1001, 2048, 7168, 8200, 34000])
@pytest.mark.parametrize("slots,gate_group", [(1, 0), (9, 1), (7, 3), (2, 64), (80, 1 << 20)])
def test_combine_norm(d, slots, gate_group, dtype):
    gen = torch.Generator().manual_seed(d + slots)
    for T, train, follow in ((1, False, True), (203 if d < 9000 else 21, True, True),
                             (9, True, False)):
        u = rand(gen, T, d, std=2.0, dtype=dtype)
        ys = rand(gen, T, slots, d, dtype=dtype)
        w, wn = (rand(gen, d, mean=1.0, std=0.2, dtype=dtype) for _ in range(2))
        gate = rand(gen, -(-T // gate_group), d, mean=0.5, std=0.3,
                    dtype=dtype) if gate_group else None
        desc = moe.make_norm_desc(T, d, EPS, dtype, slots, gate_group, 0.75)
        h, y, x_next = (torch.full_like(u, float("nan")) for _ in range(3))
        y, x_next, wn = y if train else None, x_next if follow else None, wn if follow else None
        moe.moe_combine_norm(desc, u, ys, w, gate, wn, h, y, x_next)
        wh, wy, wx = block.combine_norm(f64(u), f64(ys), f64(w), f64(gate), gate_group, 0.75,
                                        f64(wn), desc.eps)
        g = block.gate_rows(f64(gate), gate_group, T)
        # y sums terms of either sign: its error is relative to their magnitudes, and so are the
        # errors of what follows from it
        ymag = np.abs(f64(ys)).sum(1)
        hmag = np.abs(0.75 * f64(u)) + np.abs(g * f64(w)) * ymag * block.inv_rms(wy, desc.eps)
        close("h", h, wh, hmag, dtype)
        if train:
            close("y", y, wy, ymag, dtype)
        if follow:
            close("x_next", x_next, wx, np.abs(f64(wn)) * block.inv_rms(wh, desc.eps) *
                  (hmag + np.abs(wh)), dtype)
    assert moe.moe_last_device_status() == moe.OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate_group", GATES)
@pytest.mark.parametrize("d", [8, 264, 520, 1001, 2048, 5120, 8200])
def test_combine_norm_backward(d, gate_group, dtype):
    gen = torch.Generator().manual_seed(d + gate_group)
    for T in (1, 50, 2003 if d < 3000 else 700):
        y, dh = rand(gen, T, d, std=0.5, dtype=dtype), rand(gen, T, d, dtype=dtype)
        w = rand(gen, d, mean=1.0, std=0.2, dtype=dtype)
        n_gate = -(-T // gate_group) if gate_group else 0
        gate = rand(gen, n_gate, d, mean=0.5, std=0.3, dtype=dtype) if n_gate else None
        dgate = torch.full_like(gate, float("nan")) if n_gate else None
        dy = torch.full_like(y, float("nan"))
        dw = torch.full((d,), float("nan"), device="cuda")
        desc = moe.make_norm_desc(T, d, EPS, dtype, 1, gate_group)
        ws = moe.norm_backward_workspace(desc).fill_(0xff)
        moe.moe_combine_norm_backward(desc, y, w, gate, dh, dy, dw, dgate, ws)
        want, want_w, want_g = block.combine_norm_backward(f64(y), f64(w), f64(gate), gate_group,
                                                           f64(dh), desc.eps)
        g = block.gate_rows(f64(gate), gate_group, T)
        r = block.inv_rms(f64(y), desc.eps)
        c = np.abs(f64(dh) * g * f64(w))
        close("dy", dy, want, r * c + np.abs(f64(y)) * r ** 3 *
              np.mean(np.abs(f64(y)) * c, -1, keepdims=True), dtype)
        sums_close("dw", dw, want_w, np.sum(np.abs(f64(dh) * g * f64(y) * r), 0), T)
        if n_gate:
            mag = np.zeros_like(want_g)
            np.add.at(mag, np.arange(T) // gate_group, np.abs(f64(dh) * f64(w) * f64(y) * r))
            sums_close("dgate", dgate, want_g, mag, T, dtype)
        again = [t.clone() for t in (dy, dw)] + ([dgate.clone()] if n_gate else [])
        moe.moe_combine_norm_backward(desc, y, w, gate, dh, dy, dw, dgate, ws)
        for a, b in zip(again, (dy, dw, dgate)):
            assert torch.equal(a, b), "two runs differ"
    assert moe.moe_last_device_status() == moe.OK


def test_zero_rows_infinities_and_nan_stay_in_their_rows():
    T, d = 6, 512
    gen = torch.Generator().manual_seed(1)
    x, w = rand(gen, T, d), rand(gen, d, mean=1.0, std=0.1)
    x[1] = 0
    x[2, 5] = float("inf")
    x[3, 7] = float("nan")
    desc = moe.make_norm_desc(T, d, EPS)
    out = torch.empty_like(x)
    moe.moe_norm(desc, x, w, out)
    assert (out[1] == 0).all() and out[3].isnan().all() and out[2, 5].isnan()
    keep = [0, 4, 5]
    want = block.norm(f64(x)[keep], f64(w), desc.eps)
    close("out", out[keep], want, np.abs(want), "bf16")
    # a zero row has the gradient c / sqrt(eps)
    dout = rand(gen, T, d)
    dx, dw = torch.empty_like(x), torch.empty(d, device="cuda")
    moe.moe_norm_backward(desc, x, w, dout, None, dx, dw, moe.norm_backward_workspace(desc))
    want = f64(dout[1]) * f64(w) / np.sqrt(desc.eps)
    close("dx of the zero row", dx[1], want, np.abs(want), "bf16")
    assert dx[3].isnan().all()


def test_no_tokens():
    d = 256
    desc = moe.make_norm_desc(0, d, EPS, gate_group=4)
    e = torch.empty(0, d, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((d,), 7.0, device="cuda")
    moe.moe_norm(desc, e, w, e)
    ws = moe.norm_backward_workspace(desc)
    moe.moe_norm_backward(desc, e, w, e, None, e, dw, ws)
    assert (dw == 0).all()


def test_graph_and_side_stream():
    T, d = 300, 2048
    gen = torch.Generator().manual_seed(3)
    y, dh, w = rand(gen, T, d), rand(gen, T, d), rand(gen, d, mean=1.0, std=0.1)
    gate = rand(gen, 3, d, mean=0.5, std=0.1)
    desc = moe.make_norm_desc(T, d, EPS, gate_group=128)
    outs = [(torch.empty_like(y), torch.empty(d, device="cuda"), torch.empty_like(gate))
            for _ in range(2)]
    ws = [moe.norm_backward_workspace(desc) for _ in range(2)]
    moe.moe_combine_norm_backward(desc, y, w, gate, dh, *outs[0], ws[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        moe.moe_combine_norm_backward(desc, y, w, gate, dh, *outs[1], ws[1])
    for o in outs[1]:
        o.fill_(float("nan"))
    dh_new = rand(gen, T, d)
    dh.copy_(dh_new)
    graph.replay()
    moe.moe_combine_norm_backward(desc, y, w, gate, dh, *outs[0], ws[0])
    torch.cuda.synchronize()
    for a, b in zip(*outs):
        assert torch.equal(a, b)


# many tokens: rows of 128 vectors, one, two and four vectors a thread, a last thread without any,
# rows that begin and end inside a vector
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [1024, 1032, 2056, 5120, 8192, 257, 1001, 7935])
@pytest.mark.parametrize("slots,gate_group", [(1, 0), (9, 700), (2, 1)])
def test_combine_norm_of_many_tokens(d, slots, gate_group, dtype):
    gen = torch.Generator(device="cuda").manual_seed(d + slots)
    T = 1301 if d < 4000 else 1185

    def draw(*shape, std=1.0, mean=0.0):
        x = torch.randn(*shape, generator=gen, device="cuda") * std + mean
        return x.to(TYPES[dtype])

    u, ys = draw(T, d, std=2.0), draw(T, slots, d)
    w, wn = draw(d, mean=1.0, std=0.2), draw(d, mean=1.0, std=0.2)
    gate = draw(-(-T // gate_group), d, mean=0.5, std=0.3) if gate_group else None
    desc = moe.make_norm_desc(T, d, EPS, dtype, slots, gate_group, 0.75)
    h, y, x_next = (torch.full_like(u, float("nan")) for _ in range(3))
    moe.moe_combine_norm(desc, u, ys, w, gate, wn, h, y, x_next)
    wh, wy, wx = block.combine_norm(f64(u), f64(ys), f64(w), f64(gate), gate_group, 0.75, f64(wn),
                                    desc.eps)
    g = block.gate_rows(f64(gate), gate_group, T)
    ymag = np.abs(f64(ys)).sum(1)
    hmag = np.abs(0.75 * f64(u)) + np.abs(g * f64(w)) * ymag * block.inv_rms(wy, desc.eps)
    close("y", y, wy, ymag, dtype)
    close("h", h, wh, hmag, dtype)
    close("x_next", x_next, wx, np.abs(f64(wn)) * block.inv_rms(wh, desc.eps) *
          (hmag + np.abs(wh)), dtype)
    again = torch.full_like(h, float("nan"))
    moe.moe_combine_norm(desc, u, ys, w, gate, None, again, None, None)
    assert torch.equal(again, h)
    assert moe.moe_last_device_status() == moe.OK
