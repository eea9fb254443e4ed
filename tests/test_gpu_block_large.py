"""The operators around the layer on arrays of more than 2^31 elements: what the call leaves at the
far end is, bit for bit, what a call on the far end alone leaves (rows, and elements of the AdamW
step, do not depend on the rest), or for column sums what fp64 sums give.

Tolerance of the column sums: chains of fp32 additions as derived in test_gpu_block_ranges.py,
2^-24 (T / 74 + 100) of the sum of magnitudes; a bf16 gradient adds half a step.
"""
import gc

import pytest
import torch

import forward_moe_route_b200 as moe
from test_gpu_block_norm import EPS

pytestmark = pytest.mark.gpu

BF = dict(dtype=torch.bfloat16, device="cuda")
TAIL = 2000


@pytest.fixture(autouse=True)
def release():
    yield
    gc.collect()
    torch.cuda.empty_cache()


def draw(gen, *shape, std=1.0, mean=0.0):
    return torch.empty(*shape, **BF).normal_(mean, std, generator=gen)


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("T,d", [(400_003, 7168), (2_200_001, 1001)])
def test_norm(T, d):
    assert T * d > 2 ** 31
    gen = generator(d)
    x, w = draw(gen, T, d, std=2.0), draw(gen, d, mean=1.0, std=0.1)
    out, tail = torch.zeros_like(x), torch.empty(TAIL, d, **BF)
    at = (T - TAIL) // 8 * 8    # the tail starts at a multiple of 16 bytes, as a tensor does
    moe.moe_norm(moe.make_norm_desc(T, d, EPS), x, w, out)
    moe.moe_norm(moe.make_norm_desc(TAIL, d, EPS), x[at:at + TAIL], w, tail)
    assert torch.equal(out[at:at + TAIL], tail)
    assert moe.moe_last_device_status() == moe.OK


def test_end_of_a_block():
    T, d, S = 70_008, 7168, 9
    assert T * S * d > 2 ** 32
    gen = generator(1)
    u, ys, gate = draw(gen, T, d, std=2.0), draw(gen, T, S, d), draw(gen, T, d, mean=0.5, std=0.2)
    w, wn = (draw(gen, d, mean=1.0, std=0.1) for _ in range(2))
    desc, small = (moe.make_norm_desc(n, d, EPS, "bf16", S, 1, 0.5) for n in (T, TAIL))
    whole = [torch.zeros(T, d, **BF) for _ in range(3)]
    tail = [torch.empty(TAIL, d, **BF) for _ in range(3)]
    moe.moe_combine_norm(desc, u, ys, w, gate, wn, *whole)
    end = slice(T - TAIL, T)
    moe.moe_combine_norm(small, u[end], ys[end], w, gate[end], wn, *tail)
    for a, b in zip(whole, tail):
        assert torch.equal(a[end], b)
    assert moe.moe_last_device_status() == moe.OK


def sums(rows, step, T):
    """fp64 sums of f(slice) and of its magnitudes over the rows."""
    total = size = 0
    for a in range(0, T, step):
        t = rows(slice(a, min(T, a + step)))
        total, size = total + t.sum(0), size + t.abs().sum(0)
    return total, size


def test_backward_before_the_layer():
    T, d = 300_008, 7168
    assert T * d > 2 ** 31
    gen = generator(2)
    x, dout, dh = draw(gen, T, d, std=2.0), draw(gen, T, d), draw(gen, T, d)
    w = draw(gen, d, mean=1.0, std=0.1)
    dx, dw = torch.zeros_like(x), torch.empty(d, device="cuda")
    desc, small = moe.make_norm_desc(T, d, EPS), moe.make_norm_desc(TAIL, d, EPS)
    moe.moe_norm_backward(desc, x, w, dout, dh, dx, dw, moe.norm_backward_workspace(desc))
    end = slice(T - TAIL, T)
    tail, part = torch.empty(TAIL, d, **BF), torch.empty(d, device="cuda")
    moe.moe_norm_backward(small, x[end], w, dout[end], dh[end], tail, part,
                          moe.norm_backward_workspace(small))
    assert torch.equal(dx[end], tail)

    def rows(s):
        v = x[s].double()
        return dout[s].double() * v * (v.square().mean(1, keepdim=True) + desc.eps).rsqrt()

    want, size = sums(rows, 10_000, T)
    assert ((dw.double() - want).abs() <= 2.0 ** -24 * (T / 74 + 100) * size).all()
    assert moe.moe_last_device_status() == moe.OK


@pytest.mark.parametrize("group", [1, 3, 1000])
def test_backward_of_the_end_of_a_block(group):
    T, d = 300_000, 7168
    gen = generator(group)
    y, dh = draw(gen, T, d, std=0.5), draw(gen, T, d)
    w, gate = draw(gen, d, mean=1.0, std=0.1), draw(gen, T // group, d, mean=0.5, std=0.2)
    desc = moe.make_norm_desc(T, d, EPS, gate_group=group)
    dy, dgate, dw = torch.zeros_like(y), torch.zeros_like(gate), torch.empty(d, device="cuda")
    moe.moe_combine_norm_backward(desc, y, w, gate, dh, dy, dw, dgate,
                                  moe.norm_backward_workspace(desc))

    def terms(s):
        v = y[s].double()
        n = v * (v.square().mean(1, keepdim=True) + desc.eps).rsqrt()
        at = torch.arange(s.start, s.stop, device="cuda") // group
        return dh[s].double() * n, gate[at].double()

    want, size = sums(lambda s: torch.mul(*terms(s)), 10_000, T)
    chain = 2.0 ** -24 * (T / 74 + 100)
    assert ((dw.double() - want).abs() <= chain * size).all()
    # the last gate rows, and the last rows
    k = 3000 // group
    end = slice(T - k * group, T)
    t = (terms(end)[0] * w.double()).view(k, group, d)
    want, size = t.sum(1), t.abs().sum(1)
    assert ((dgate[-k:].double() - want).abs() <= 2.0 ** -8 * want.abs() + chain * size).all()
    small = moe.make_norm_desc(k * group, d, EPS, gate_group=group)
    tail, part, g = (torch.empty(k * group, d, **BF), torch.empty(d, device="cuda"),
                     torch.empty(k, d, **BF))
    moe.moe_combine_norm_backward(small, y[end], w, gate[-k:], dh[end], tail, part, g,
                                  moe.norm_backward_workspace(small))
    assert torch.equal(dy[end], tail)
    assert moe.moe_last_device_status() == moe.OK


def test_products_of_many_rows():
    R, d_in, d_out = 540_011, 64, 4096
    assert R * d_out > 2 ** 31
    gen = generator(4)
    x, dy, w = draw(gen, R, d_in), draw(gen, R, d_out), draw(gen, 3, d_out, d_in, std=0.1)
    cut = R - 777
    cut -= cut % 8
    offsets = torch.tensor([0, 5, cut, R], dtype=torch.int32, device="cuda")
    tail = torch.tensor([0, R - cut], dtype=torch.int32, device="cuda")
    y, y_tail = torch.zeros(R, d_out, **BF), torch.empty(R - cut, d_out, **BF)
    moe.moe_grouped_mm(x, w, offsets, y)
    moe.moe_grouped_mm(x[cut:], w[2:], tail, y_tail)
    assert torch.equal(y[cut:], y_tail)
    dx, dx_tail = torch.zeros(R, d_in, **BF), torch.empty(R - cut, d_in, **BF)
    moe.moe_grouped_mm_dx(dy, w, offsets, dx)
    moe.moe_grouped_mm_dx(dy[cut:], w[2:], tail, dx_tail)
    assert torch.equal(dx[cut:], dx_tail)
    dw, dw_tail = torch.zeros(3, d_out, d_in, device="cuda"), torch.empty(1, d_out, d_in,
                                                                          device="cuda")
    moe.moe_grouped_mm_dw(dy, x, offsets, dw)
    moe.moe_grouped_mm_dw(dy[cut:], x[cut:], tail, dw_tail)
    assert torch.equal(dw[2], dw_tail[0])
    assert moe.moe_last_device_status() == moe.OK


@pytest.mark.parametrize("rows", [3, 300])
def test_products_of_many_weights(rows):
    G, d_in, d_out = 400, 1408, 4096
    assert G * d_in * d_out > 2 ** 31
    gen = generator(5)
    x, dy, w = draw(gen, rows, d_in), draw(gen, rows, d_out), draw(gen, G, d_out, d_in, std=0.1)
    offsets = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    offsets[-1] = rows
    last = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    y, y_last = torch.zeros(rows, d_out, **BF), torch.empty(rows, d_out, **BF)
    moe.moe_grouped_mm(x, w, offsets, y)
    moe.moe_grouped_mm(x, w[-1:].clone(), last, y_last)
    want = x.double() @ w[-1].double().T
    size = x.double().abs() @ w[-1].double().abs().T
    for got in (y, y_last):         # a call of few rows may take another kernel than the other
        tol = 2.0 ** -8 * want.abs() + (d_in / 16 + 17) * 2.0 ** -23 * size
        assert ((got.double() - want).abs() <= tol).all()
    dx, dx_last = torch.zeros(rows, d_in, **BF), torch.empty(rows, d_in, **BF)
    moe.moe_grouped_mm_dx(dy, w, offsets, dx)
    moe.moe_grouped_mm_dx(dy, w[-1:].clone(), last, dx_last)
    assert torch.equal(dx, dx_last)
    del w
    for kind in (torch.float32, torch.bfloat16):
        dw = torch.full((G, d_out, d_in), 7.0, dtype=kind, device="cuda")
        one = torch.empty(1, d_out, d_in, dtype=kind, device="cuda")
        moe.moe_grouped_mm_dw(dy, x, offsets, dw)
        moe.moe_grouped_mm_dw(dy, x, last, one)
        assert torch.equal(dw[-1], one[0])
        assert int(torch.count_nonzero(dw[:-1])) == 0
        del dw
    assert moe.moe_last_device_status() == moe.OK


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw(bits):
    n = 2 ** 31 + 4099
    gen = generator(bits)
    p = torch.empty(n, device="cuda").normal_(0, 0.1, generator=gen)
    g, copy = draw(gen, n, std=1e-2), torch.zeros(n, **BF)
    if bits == 32:
        m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
        scales = {}
    else:
        m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
        scales = {k: [torch.zeros(-(-n // 128), device="cuda")] for k in ("m_scale", "v_scale")}
    end = slice(n - 4099 - 2048, n)
    q, few = p[end].clone(), {k: [x[0][end.start // 128:].clone()] for k, x in scales.items()}
    state = [t[end].clone() for t in (m, v, copy)]
    desc = moe.make_adamw_desc(1e-2, state_bits=bits, seed=3)
    moe.moe_adamw(desc, moe.adamw_table([p], [g], [m], [v], p_bf16=[copy], **scales), 1)
    moe.moe_adamw(desc, moe.adamw_table([q], [g[end].clone()], [state[0]], [state[1]],
                                        p_bf16=[state[2]], **few), 1)
    assert torch.equal(p[end], q) and torch.equal(copy[end], state[2])
    assert moe.moe_last_device_status() == moe.OK
    if bits == 32:
        assert torch.equal(m[end], state[0]) and torch.equal(v[end], state[1])
        return
    for k, x in scales.items():
        assert torch.equal(x[0][end.start // 128:], few[k][0])
    # the codes are drawn by an element's place: one code apart at most, and not all the same
    for a, b in ((m[end], state[0]), (v[end], state[1])):
        assert (a.int() - b.int()).abs().max() <= 1 and not torch.equal(a, b)
