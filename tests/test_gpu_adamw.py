"""GPU parity of the AdamW step with the fp64 oracle.

Tolerances, from the arithmetic (u = 2^-24).  m' = b1 m + (1 - b1) g: two rounded constants, one
rounded product, one rounding of the sum: 4 u (|b1 m| + |(1 - b1) g|).  v' the same with g^2
rounded too: 5 u v'.  The root and the quotient are the hardware's approximations (2 u and 4 u) of
factors that carry 3 u each at most: the move of p is right to 16 u + the error of m' it carries,
so 24 u of lr / (1 - b1^t) (|b1 m| + |(1 - b1) g|) / (sqrt + eps); p' itself adds a rounding of p' and
of the decay factor, 2 u |p|.  8-bit moments add a product with the scale (and a square for v): 3 u
more of each.  A bf16 copy is p' rounded once: 2^-8.
"""
import numpy as np
import pytest
import torch

import forward_moe_route_b200 as moe
from oracle import block

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8)


def f64(t):
    return t.double().cpu().numpy()


class State:
    """A list of tensors with moments as a few steps leave them; `shift` elements off alignment."""

    def __init__(self, sizes, bits, grads, seed=0, shift=0, copies=True):
        gen = torch.Generator().manual_seed(seed)
        self.bits, self.sizes = bits, sizes

        def put(x):
            room = torch.zeros(len(x) + shift + 1, dtype=x.dtype, device="cuda")
            room[shift:shift + len(x)] = x.cuda()
            return room[shift:shift + len(x)]

        def draw(n, std):
            return torch.randn(n, generator=gen) * std

        self.p = [put(draw(n, 0.1)) for n in sizes]
        self.g = [put(draw(n, 1e-2).to(torch.bfloat16 if grads == "bf16" else torch.float32))
                  for n in sizes]
        self.pb = [put(torch.zeros(n, dtype=torch.bfloat16)) if copies else None for n in sizes]
        if bits == 32:
            self.m = [put(draw(n, 3e-3)) for n in sizes]
            self.v = [put(draw(n, 6e-3).square()) for n in sizes]
            self.ms = self.vs = None
        else:
            def codes(n):
                return torch.randint(0, 0x7f, (n,), generator=gen, dtype=torch.uint8)
            self.m = [put((codes(n) | (codes(n) << 7)).view(torch.float8_e4m3fn)) for n in sizes]
            self.v = [put(codes(n).view(torch.float8_e4m3fn)) for n in sizes]
            self.ms = [put(draw(-(-n // 128), 2e-5).abs()) for n in sizes]
            self.vs = [put(draw(-(-n // 128), 4e-5).abs() + 1e-6) for n in sizes]

    def table(self, decay=0.1):
        return moe.adamw_table(self.p, self.g, self.m, self.v, p_bf16=self.pb, weight_decay=decay,
                               m_scale=self.ms, v_scale=self.vs)

    def tensors(self):
        out = self.p + self.m + self.v + [x for x in self.pb if x is not None]
        return out + (self.ms + self.vs if self.ms else [])

    def moments(self, i):
        """m and v of tensor i in fp64."""
        if self.bits == 32:
            return f64(self.m[i]), f64(self.v[i])
        n = self.sizes[i]
        value = [block.e4m3_value(c[i].view(torch.uint8).cpu().numpy()) for c in (self.m, self.v)]
        return (value[0] * block.spread(f64(self.ms[i]), n),
                (value[1] * block.spread(f64(self.vs[i]), n)) ** 2)


def within(name, got, want, tol):
    off = np.abs(got - want) - tol
    assert np.isfinite(got).all(), name
    assert (off <= 1e-36).all(), f"{name}: over by {off.max():.3e} at {np.argmax(off)}"


def one_step(s, table, step, decays, seed=0):
    """Run a step and hold every tensor against the oracle's step from the state before."""
    desc = moe.make_adamw_desc(**HYPER, state_bits=s.bits, seed=seed)
    before = [(f64(s.p[i]), f64(s.g[i]), *s.moments(i)) for i in range(len(s.sizes))]
    moe.moe_adamw(desc, table, step)
    assert moe.moe_last_device_status() == moe.OK
    b1, b2 = HYPER["beta1"], HYPER["beta2"]
    extra = 0 if s.bits == 32 else 3
    for i, (p, g, m, v) in enumerate(before):
        n = s.sizes[i]
        wp, wm, wv = block.adamw(p, g, m, v, step, decay=decays[i], **HYPER)
        mag = np.abs(b1 * m) + np.abs((1 - b1) * g)
        down = np.sqrt(wv / (1 - b2 ** step)) + HYPER["eps"]
        tol_p = (24 + extra) * U * HYPER["lr"] / (1 - b1 ** step) * mag / down + 2 * U * (
            np.abs(p) + np.abs(wp))
        within("p", f64(s.p[i]), wp, tol_p)
        if s.pb[i] is not None:
            assert torch.equal(s.pb[i], s.p[i].to(torch.bfloat16))
        if s.bits == 32:
            within("m", f64(s.m[i]), wm, 4 * U * mag)
            within("v", f64(s.v[i]), wv, 5 * U * wv)
            continue
        root = np.sqrt(wv)
        words = block.random_words(n, i, seed, step)
        for name, codes, scales, x, err, bits in (
                ("m", s.m, s.ms, wm, 7 * U * mag, words & np.uint64(0xffff)),
                ("v", s.v, s.vs, root, 8 * U * root, words >> np.uint64(16))):
            held = f64(scales[i])
            most = block.block_scales(x)
            within(name + "_scale", held, most, 2 * U * most + block.block_scales(err))
            c = codes[i].view(torch.uint8).cpu().numpy().astype(np.int64)
            inv = np.where(held > 0, 1 / np.where(held > 0, held, 1), 0)
            at = np.minimum(np.abs(x) * block.spread(inv, n), 448.0)
            place = block.e4m3_position(at) + bits / 65536.0
            want = np.minimum(np.floor(place), 0x7e)
            if name == "v":
                want = np.where((want == 0) & (x > 0), 1, want)
            # x / scale carries the error of x, of the inverse scale and of their product; a code
            # step is at least 1/16 of the value, and the kernel compares 20 bits of a step
            slack = 16 * (err / np.maximum(np.abs(x), 1e-30) + 4 * U) + 2.0 ** -19
            near = np.abs(place - np.round(place)) <= slack
            same = (c & 0x7f) == want
            assert (same | near).all(), f"{name}: codes differ at {np.argmin(same | near)}"
            assert (np.abs((c & 0x7f) - want) <= 1).all()
            sign = (c & 0x80) != 0
            assert (sign == (x < 0))[np.abs(x) > err].all()


SIZES = [1, 7, 8, 9, 127, 128, 129, 1000, 2047, 2048, 2049, 20011]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grads", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [0, 1, 2, 8])
def test_steps(bits, grads, shift):
    s = State(SIZES, bits, grads, seed=shift, shift=shift)
    decays = [0.1 * (i % 3) for i in range(len(SIZES))]
    table = s.table(decays)
    decays = [float(np.float32(x)) for x in decays]
    for step in (1, 2, 3, 1000):
        one_step(s, table, step, decays, seed=12345678901234 + shift)


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors_some_empty_and_no_copies(bits):
    sizes = [(i * 37) % 400 for i in range(700)]
    s = State(sizes, bits, "f32", copies=False)
    one_step(s, s.table(0.0), 5, [0.0] * len(sizes))


def test_neighbours_of_a_tensor_stay():
    """Tensors packed into flat buffers without gaps: elements around a tensor are left alone."""
    gen = torch.Generator().manual_seed(4)
    flat = {k: torch.randn(5000, generator=gen).abs().cuda() for k in "pgmv"}
    keep = {k: x.clone() for k, x in flat.items()}
    cut = {k: [x[3:1003], x[1003:1004], x[2000:4999]] for k, x in flat.items()}
    table = moe.adamw_table(cut["p"], cut["g"], cut["m"], cut["v"])
    moe.moe_adamw(moe.make_adamw_desc(**HYPER), table, 1)
    inside = torch.zeros(5000, dtype=torch.bool, device="cuda")
    for a, b in ((3, 1003), (1003, 1004), (2000, 4999)):
        inside[a:b] = True
    for k in "pmv":
        assert torch.equal(flat[k][~inside], keep[k][~inside])
        assert (flat[k][inside] != keep[k][inside]).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_zero_start_and_zero_gradients(bits):
    s = State([300, 77], bits, "bf16")
    for x in s.m + s.v + (s.ms + s.vs if bits == 8 else []):
        x.zero_()
    s.g[1].zero_()
    p1 = f64(s.p[1])
    one_step(s, s.table(0.0), 1, [0.0, 0.0])
    np.testing.assert_array_equal(f64(s.p[1]), p1)
    m, v = s.moments(1)
    assert (m == 0).all() and (v == 0).all()
    # gradients that are gone: a positive root is not held as zero
    s.g[0].zero_()
    for step in range(2, 12):
        one_step(s, s.table(0.0), step, [0.0, 0.0], seed=step)
    assert (s.moments(0)[1] > 0).all() or bits == 32


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_gradients_show(bits, bad):
    s = State([512], bits, "f32")
    s.g[0][200] = bad
    before = f64(s.p[0])
    moe.moe_adamw(moe.make_adamw_desc(**HYPER, state_bits=bits), s.table(0.0), 2)
    assert not np.isfinite(f64(s.p[0])[200])
    m, v = s.moments(0)
    assert not np.isfinite(m[200]) and not np.isfinite(v[200])
    rest = np.r_[0:128, 256:512]
    assert np.isfinite(f64(s.p[0])[rest]).all() and np.isfinite(m[rest]).all()
    assert (f64(s.p[0])[rest] != before[rest]).any()


def test_rounding_is_unbiased():
    """The mean of decoded - x over elements with the same distance to the code below."""
    n = 1 << 20
    s = State([n], 8, "f32")
    for x in (s.m[0], s.v[0]):
        x.view(torch.uint8).zero_()
    # m' = (1 - b1) g: 448 units of 1 / 448 in each block, the rest at 0.3 of a code step
    s.g[0].copy_(torch.full((n,), 17.3 / 16))
    s.g[0][::128] = 448 / 256.0
    moe.moe_adamw(moe.make_adamw_desc(**HYPER, state_bits=8, seed=3), s.table(), 1)
    m, _ = s.moments(0)
    x = 0.1 * f64(s.g[0])
    keep = np.arange(n) % 128 != 0
    step = np.ptp(m[keep])
    assert 0 < step < 0.13 * x[1]
    frac = (x[1] - m[keep].min()) / step
    sigma = step * np.sqrt(frac * (1 - frac) / keep.sum())
    assert abs(m[keep].mean() - x[1]) < 5 * sigma + 2.0 ** -16 * step


@pytest.mark.parametrize("bits", [32, 8])
def test_graph_follows_step_and_lr_on_the_device(bits):
    a, b = (State([1000, 4097], bits, "bf16", seed=2) for _ in range(2))
    desc = moe.make_adamw_desc(**HYPER, state_bits=bits, seed=9)
    ta, tb = a.table(), b.table()
    step = torch.zeros(1, dtype=torch.int32, device="cuda")
    lr = torch.zeros(1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_adamw(desc, ta, step, lr=lr)
    for k in (1, 2, 3, 77):
        step.fill_(k)
        lr.fill_(1e-3 * k)
        graph.replay()
        now = moe.make_adamw_desc(**{**HYPER, "lr": float(np.float32(1e-3 * k))}, state_bits=bits,
                                  seed=9)
        moe.moe_adamw(now, tb, k)
        for x, y in zip(a.tensors(), b.tensors()):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), k
    # the step number counts from 1: anything below is reported and changes nothing
    keep = [x.clone() for x in a.tensors()]
    step.fill_(0)
    graph.replay()
    assert moe.moe_last_device_status() == moe.ERR_DEVICE_CHECK
    for x, y in zip(a.tensors(), keep):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_a_table_of_the_other_states_is_reported():
    s = State([300], 32, "f32")
    t = s.table()
    t.state_bits = 8
    keep = [x.clone() for x in s.tensors()]
    moe.moe_adamw(moe.make_adamw_desc(**HYPER, state_bits=8), t, 1)
    assert moe.moe_last_device_status() == moe.ERR_DEVICE_CHECK
    for x, y in zip(s.tensors(), keep):
        assert torch.equal(x, y)
