"""The operators around the layer where their kernels take another course than at small sizes:
AdamW chunks of several spans, gate rows of a few tokens by the thousand, rows so long that one of
them fills a block's ring, and rows beyond a block's registers with gates.

Tolerances of the norms.  bf16 outputs: half a step, 2^-8, of the value and 2^-19 of the sum of the
magnitudes behind it for the fp32 arithmetic, as in test_gpu_block_norm.py.  Column sums: a chain of
n fp32 additions errs by at most n 2^-24 of the sum of magnitudes M, a term carries fewer than 16
roundings.  A block takes its share of the T rows, 148 blocks or more when there are as many units
(four for each of them at most, so at most twice the mean), else a unit of at most ceil(T / units)
rows; its row groups' sums (16 at most) are joined, then those of the blocks, in 32 slices of at
most 592 / 32 + 1 rows.  So n <= 2 T / 148 + 16 + 16 + 20 + 32 wherever units are at least as many
as blocks, and 2^-24 (T / 74 + 100) M is used; units are fewer only where T is below 148 rows a
block, and then no chain is longer than those 100.
"""
import numpy as np
import pytest
import torch

import forward_moe_route_b200 as moe
from oracle import block

pytestmark = pytest.mark.gpu

EPS = 1e-5
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def hold(name, got, want, tol):
    off = np.abs(f64(got) - want) - tol
    assert np.isfinite(off).all() and (off <= 1e-30).all(), f"{name}: over by {off.max():.3e}"


def half(dtype):
    return 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24


# (d, gate_group, T).  A gate row for 2 or 3 tokens, in more units than the row groups of 148
# blocks take at once (16 groups a block at 64 columns, 4 at 4096); whole gate rows whose sums leave
# room for one stage in the ring (bf16: 188 of 8 rows of 8192, 150 of 2 rows of 16384); the looping
# kernel with vectors and with single elements
CASES = [(64, 3, 16001), (264, 3, 8000), (520, 2, 5003), (1001, 2, 2600), (4096, 2, 2500),
         (8192, 2, 300), (8192, 8, 1500), (8192, 64, 1500), (8192, 1, 200), (8192, 1 << 20, 333), (16384, 2, 300),
         (16384, 700, 333), (16392, 3, 50), (20001, 64, 150), (16392, 1 << 20, 40),
         (9001, 1, 40), (4096, 1024, 2500)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,gate_group,T", CASES)
def test_end_of_block_backward(d, gate_group, T, dtype):
    gen = torch.Generator(device="cuda").manual_seed(d + gate_group + T)

    def draw(*shape, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std + mean).to(TYPES[dtype])

    y, dh, w = draw(T, d, std=0.5), draw(T, d), draw(d, std=0.2, mean=1.0)
    gate = draw(-(-T // gate_group), d, std=0.3, mean=0.5)
    desc = moe.make_norm_desc(T, d, EPS, dtype, 1, gate_group)
    dy, dgate = torch.full_like(y, float("nan")), torch.full_like(gate, float("nan"))
    dw = torch.full((d,), float("nan"), device="cuda")
    ws = moe.norm_backward_workspace(desc).fill_(0xff)
    moe.moe_combine_norm_backward(desc, y, w, gate, dh, dy, dw, dgate, ws)
    assert moe.moe_last_device_status() == moe.OK
    Y, DH, W, G = f64(y), f64(dh), f64(w), f64(gate)
    want, want_w, want_g = block.combine_norm_backward(Y, W, G, gate_group, DH, desc.eps)
    rows = block.gate_rows(G, gate_group, T)
    n = np.abs(Y) * block.inv_rms(Y, desc.eps)
    c = np.abs(DH * rows * W)
    size = block.inv_rms(Y, desc.eps) * (c + n * np.mean(n * c, -1, keepdims=True))
    hold("dy", dy, want, half(dtype) * np.abs(want) + 2.0 ** -19 * size)
    chain = 2.0 ** -24 * (T / 74 + 100)
    hold("dw", dw, want_w, 2.0 ** -24 * np.abs(want_w) + chain * np.sum(np.abs(DH * rows) * n, 0))
    size = np.zeros_like(want_g)
    np.add.at(size, np.arange(T) // gate_group, np.abs(DH * W) * n)
    hold("dgate", dgate, want_g, half(dtype) * np.abs(want_g) + chain * size)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,T", [(64, 70001), (8192, 700), (16384, 400), (24576, 200), (2048, 1)])
def test_backward_before_the_layer(d, T, dtype):
    gen = torch.Generator(device="cuda").manual_seed(d + T)

    def draw(*shape, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std + mean).to(TYPES[dtype])

    x, dout, dh, w = draw(T, d, std=2.0), draw(T, d), draw(T, d), draw(d, std=0.2, mean=1.0)
    desc = moe.make_norm_desc(T, d, EPS, dtype, res_scale=0.5)
    dx, dw = torch.full_like(x, float("nan")), torch.full((d,), float("nan"), device="cuda")
    ws = moe.norm_backward_workspace(desc).fill_(0xff)
    moe.moe_norm_backward(desc, x, w, dout, dh, dx, dw, ws)
    assert moe.moe_last_device_status() == moe.OK
    X, UP, DH, W = f64(x), f64(dout), f64(dh), f64(w)
    want, want_w = block.norm_backward(X, W, UP, DH, 0.5, desc.eps)
    n, c = np.abs(X) * block.inv_rms(X, desc.eps), np.abs(UP * W)
    size = block.inv_rms(X, desc.eps) * (c + n * np.mean(n * c, -1, keepdims=True))
    hold("dx", dx, want, half(dtype) * np.abs(want) + 2.0 ** -19 * (size + np.abs(0.5 * DH)))
    hold("dw", dw, want_w, 2.0 ** -24 * np.abs(want_w) +
         2.0 ** -24 * (T / 74 + 100) * np.sum(np.abs(UP) * n, 0))


class Moments8:
    """A list with 8-bit moments as a few steps leave them, `shift` elements off alignment."""

    def __init__(self, sizes, grads, shift, seed=7):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.sizes = sizes

        def put(x):
            room = torch.zeros(len(x) + shift, dtype=x.dtype, device="cuda")
            room[shift:].copy_(x)
            return room[shift:]

        def draw(n, std):
            return torch.randn(n, generator=gen, device="cuda") * std

        def codes(n):
            return torch.randint(0, 0x7f, (n,), generator=gen, device="cuda", dtype=torch.uint8)

        self.p = [put(draw(n, 0.1)) for n in sizes]
        self.g = [put(draw(n, 1e-2).to(TYPES[grads])) for n in sizes]
        self.pb = [put(torch.zeros(n, dtype=torch.bfloat16, device="cuda")) for n in sizes]
        self.m = [put(codes(n) | (codes(n) << 7)) for n in sizes]
        self.v = [put(codes(n)) for n in sizes]
        self.ms = [draw(-(-n // 128), 2e-5).abs() for n in sizes]
        self.vs = [draw(-(-n // 128), 4e-5).abs() + 1e-6 for n in sizes]

    def table(self, keep=None):
        """Of all tensors, or of tensor `keep` with empty ones in the others' places."""
        def of(x):
            return [t if keep in (None, i) else t[:0] for i, t in enumerate(x)]
        return moe.adamw_table(of(self.p), of(self.g), of(self.m), of(self.v), p_bf16=of(self.pb),
                               weight_decay=0.1, m_scale=of(self.ms), v_scale=of(self.vs))

    def tensors(self, i):
        return [x[i] for x in (self.p, self.pb, self.m, self.v, self.ms, self.vs)]


# chunks of 4 spans (10 to 39 million elements are 2 to 7 of them) through rings of 2 (fp32
# gradients), of 16 through rings of 3 (bf16), with tensors that end inside a span, at the end of
# one, of a chunk, and inside their first
@pytest.mark.parametrize("grads,total", [("f32", 22_000_000), ("bf16", 80_000_000)])
def test_adamw_chunks_of_several_spans(grads, total):
    spans = min(16, total // (2048 * 148 * 16))
    assert spans == (4 if grads == "f32" else 16)
    chunk = 2048 * spans
    sizes = [5 * chunk, 777, 3 * chunk + 2048, total // 2 + 13, 2 * chunk - 2048 + 128, 2048, 0]
    sizes[-1] = total - sum(sizes)
    assert sizes[-1] > 5_000_000
    whole, apart, shifted = (Moments8(sizes, grads, s) for s in (0, 0, 1))
    desc = moe.make_adamw_desc(3e-3, state_bits=8, seed=1234567)
    one, odd = whole.table(), shifted.table()
    for step in (1, 2):
        moe.moe_adamw(desc, one, step)
        moe.moe_adamw(desc, odd, step)
        # each tensor by itself, at its place in the list: fewer spans a chunk
        for i in range(len(sizes)):
            moe.moe_adamw(desc, apart.table(keep=i), step)
        assert moe.moe_last_device_status() == moe.OK
        for i in range(len(sizes)):
            for a, b, c in zip(whole.tensors(i), apart.tensors(i), shifted.tensors(i)):
                assert torch.equal(a, b), (step, i, "by itself")
                assert torch.equal(a, c), (step, i, "off alignment")
    # and with the step on the device
    moe.moe_adamw(desc, one, torch.tensor([3], dtype=torch.int32, device="cuda"))
    moe.moe_adamw(desc, odd, 3)
    assert moe.moe_last_device_status() == moe.OK
    for i in range(len(sizes)):
        for a, c in zip(whole.tensors(i), shifted.tensors(i)):
            assert torch.equal(a, c), i
    # the largest tensor's step follows the formula (fp32 p: 27 2^-24 of the move, see
    # test_gpu_adamw.py, and a rounding of p and of the decay factor)
    big = Moments8(sizes, grads, 0)
    i, n = 3, sizes[3]
    p, g = big.p[i].double(), big.g[i].double()
    value = torch.tensor(block.e4m3_value(np.arange(256, dtype=np.uint8)), device="cuda")
    m = value[big.m[i].long()] * big.ms[i].double().repeat_interleave(128)[:n]
    v = (value[big.v[i].long()] * big.vs[i].double().repeat_interleave(128)[:n]) ** 2
    moe.moe_adamw(desc, big.table(), 5)
    size = (0.9 * m).abs() + (0.1 * g).abs()
    m, v = 0.9 * m + 0.1 * g, 0.95 * v + 0.05 * g * g
    down = (v / (1 - 0.95 ** 5)).sqrt() + 1e-8
    decay = float(np.float32(0.1))
    want = p - 3e-3 * (decay * p + m / (1 - 0.9 ** 5) / down)
    tol = 2.0 ** -24 * (27 * 3e-3 / (1 - 0.9 ** 5) * size / down + 2 * (p.abs() + want.abs()))
    assert ((big.p[i].double() - want).abs() <= tol).all()
