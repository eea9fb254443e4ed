"""The operators around the layer, what needs no GPU: the fp64 oracle's
gradients against differences, and the refusals of the entry points."""
import ctypes

import numpy as np
import pytest

import forward_moe_route_b200 as moe
from oracle import block


def differences(f, x, e=1e-6):
    """df/dx of a scalar function by central differences."""
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        keep = x[i]
        x[i] = keep + e
        up = f()
        x[i] = keep - e
        down = f()
        x[i] = keep
        g[i] = (up - down) / (2 * e)
    return g


# central differences of step e = 1e-6 of functions of order 10: the rounding of f, 1e-15 * 10,
# over e leaves 1e-8, the truncation e^2 less
DIFF = 1e-6


@pytest.mark.parametrize("gate_group", [0, 1, 2, 100])
def test_oracle_norm_gradients_against_differences(gate_group):
    rng = np.random.default_rng(gate_group)
    T, d, eps, res = 5, 6, 1e-2, 0.7
    u, ys = rng.normal(size=(T, d)), rng.normal(size=(T, 3, d))
    w, wn = 1 + 0.2 * rng.normal(size=d), 1 + 0.2 * rng.normal(size=d)
    gate = rng.normal(size=(-(-T // gate_group), d)) if gate_group else None
    gh, gx = rng.normal(size=(T, d)), rng.normal(size=(T, d))

    def loss():
        h, _, xn = block.combine_norm(u, ys, w, gate, gate_group, res, wn, eps)
        return np.sum(gh * h) + np.sum(gx * xn)

    h, y, _ = block.combine_norm(u, ys, w, gate, gate_group, res, wn, eps)
    dh, dwn = block.norm_backward(h, wn, gx, gh, 1.0, eps)
    dy, dw, dgate = block.combine_norm_backward(y, w, gate, gate_group, dh, eps)
    np.testing.assert_allclose(differences(loss, u), res * dh, atol=DIFF)
    np.testing.assert_allclose(differences(loss, ys), np.repeat(dy[:, None], 3, 1), atol=DIFF)
    np.testing.assert_allclose(differences(loss, w), dw, atol=DIFF)
    np.testing.assert_allclose(differences(loss, wn), dwn, atol=DIFF)
    if gate_group:
        np.testing.assert_allclose(differences(loss, gate), dgate, atol=DIFF)


def norm_desc(**kw):
    base = dict(T=16, d=256, eps=1e-6, dtype="bf16", n_slots=2, gate_group=4, res_scale=1.0)
    base.update(kw)
    return moe.make_norm_desc(**base)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(d=0), dict(d=65537), dict(n_slots=0),
                                dict(n_slots=81), dict(gate_group=-1), dict(eps=0.0),
                                dict(eps=float("nan")), dict(eps=float("inf")),
                                dict(res_scale=float("inf"))])
def test_invalid_norm_descriptors(kw):
    d = norm_desc(**kw)
    L = moe.lib()
    assert moe.moe_norm_backward_workspace_size(d) == 0
    r = ctypes.byref(d)
    assert L.moe_norm(r, 16, 32, 48, None) == moe.ERR_INVALID_ARG
    assert L.moe_combine_norm(r, 16, 32, 48, 64, 80, 96, 112, 128, None) == moe.ERR_INVALID_ARG
    assert L.moe_norm_backward(r, 16, 32, 48, 64, 80, 96, 112, 1 << 30,
                               None) == moe.ERR_INVALID_ARG
    assert L.moe_combine_norm_backward(r, 16, 32, 48, 64, 80, 96, 112, 128, 1 << 30,
                                       None) == moe.ERR_INVALID_ARG


def test_norm_struct_matches_header_layout():
    assert ctypes.sizeof(moe.MoeNormDesc) == 7 * 4
    d = norm_desc()
    d.act_dtype = moe.DT_E4M3
    assert moe.moe_norm_backward_workspace_size(d) == 0


def test_norm_entry_points_reject_before_touching_cuda():
    L = moe.lib()
    d = norm_desc()
    r, bad = ctypes.byref(d), moe.ERR_INVALID_ARG
    plain = norm_desc(gate_group=0)
    p = ctypes.byref(plain)
    # missing, misaligned, and an output at an input's address
    assert L.moe_norm(r, None, 32, 48, None) == bad
    assert L.moe_norm(r, 16, 33, 48, None) == bad
    assert L.moe_norm(r, 16, 32, 16, None) == bad
    ok = [16, 32, 48, 64, 80, 96, 112, 128]
    for i in (0, 1, 2, 5):
        assert L.moe_combine_norm(r, *ok[:i], None, *ok[i + 1:], None) == bad, i
    for i in range(8):
        assert L.moe_combine_norm(r, *ok[:i], ok[i] + 2, *ok[i + 1:], None) == bad, i
    # a gate without gate_group, gate_group without a gate
    assert L.moe_combine_norm(p, *ok, None) == bad
    assert L.moe_combine_norm(r, 16, 32, 48, None, 80, 96, 112, 128, None) == bad
    # w_next without x_next and the other way round
    assert L.moe_combine_norm(r, 16, 32, 48, 64, None, 96, 112, 128, None) == bad
    assert L.moe_combine_norm(r, 16, 32, 48, 64, 80, 96, 112, None, None) == bad
    # outputs on inputs and on one another
    for i in range(5):
        assert L.moe_combine_norm(r, *ok[:5], ok[i], 112, 128, None) == bad, i
    assert L.moe_combine_norm(r, *ok[:5], 96, 96, 128, None) == bad
    assert L.moe_combine_norm(r, *ok[:5], 96, 112, 112, None) == bad
    # backward
    big = 1 << 30
    for i in (0, 1, 2, 4, 5):
        a = [16, 32, 48, 64, 80, 96]
        a[i] = None
        assert L.moe_norm_backward(r, *a, 112, big, None) == bad, i
    assert L.moe_norm_backward(r, 16, 32, 48, 64, 64, 96, 112, big, None) == bad
    assert L.moe_norm_backward(r, 16, 32, 48, 64, 80, 96, None, big, None) == moe.ERR_WORKSPACE
    assert L.moe_norm_backward(r, 16, 32, 48, 64, 80, 96, 112, 16, None) == moe.ERR_WORKSPACE
    assert L.moe_combine_norm_backward(r, 16, 32, None, 64, 80, 96, 112, 128, big, None) == bad
    assert L.moe_combine_norm_backward(r, 16, 32, 48, 64, 80, 96, None, 128, big, None) == bad
    assert L.moe_combine_norm_backward(p, 16, 32, 48, 64, 80, 96, 112, 128, big, None) == bad
    assert L.moe_combine_norm_backward(r, 16, 32, 48, 64, 80, 96, 48, 128, big, None) == bad
    assert L.moe_combine_norm_backward(r, 16, 32, 48, 64, 80, 96, 112, 128, 16,
                                       None) == moe.ERR_WORKSPACE


def test_norm_binding_refuses():
    import torch
    d = norm_desc(gate_group=0)
    x = torch.zeros(16, 256, dtype=torch.bfloat16)
    w = torch.zeros(256, dtype=torch.bfloat16)
    for args, what in [((x[:15], w, x), "holds"), ((x.t(), w, x), "contiguous"),
                       ((x.float(), w, x), "float32"), ((x, None, x), "missing"),
                       ((x, w, x), "CUDA")]:
        with pytest.raises(moe.MoeError, match=what) as e:
            moe.moe_norm(d, *args)
        assert e.value.status == moe.ERR_INVALID_ARG


# ---------------------------------------------------------------- grouped products
def test_oracle_grouped_gradients_against_differences():
    rng = np.random.default_rng(3)
    offsets = np.array([1, 1, 4, 6])
    x, w = rng.normal(size=(7, 3)), rng.normal(size=(3, 4, 3))
    dy = rng.normal(size=(7, 4))

    def loss():
        return np.sum(dy * block.grouped_mm(x, w, offsets, np.zeros((7, 4))))

    dx = block.grouped_mm_dx(dy, w, offsets, np.zeros_like(x))
    dw = block.grouped_mm_dw(dy, x, offsets, np.zeros_like(w))
    np.testing.assert_allclose(differences(loss, x), dx, atol=DIFF)
    np.testing.assert_allclose(differences(loss, w), dw, atol=DIFF)


def test_grouped_entry_points_reject_before_touching_cuda():
    L, bad = moe.lib(), moe.ERR_INVALID_ARG
    ok = (4, 16, 64, 128)
    for dims in [(0, 16, 64, 128), (1025, 16, 64, 128), (4, -1, 64, 128), (4, 16, 0, 128),
                 (4, 16, 68, 128), (4, 16, 64, 4), (4, 16, 64, 65544), (4, 16, 65544, 64)]:
        assert L.moe_grouped_mm(*dims, 16, 32, 48, 64, None) == bad, dims
        assert L.moe_grouped_mm_dx(*dims, 16, 32, 48, 64, None) == bad, dims
        assert L.moe_grouped_mm_dw(*dims, 16, 32, 48, 64, 0, 0, None) == bad, dims
    for i in range(4):
        for wrong in (None, 40):
            p = [16, 32, 48, 64]
            p[i] = wrong
            assert L.moe_grouped_mm(*ok, *p, None) == bad
            assert L.moe_grouped_mm_dx(*ok, *p, None) == bad
            assert L.moe_grouped_mm_dw(*ok, *p, 0, 0, None) == bad
    for i in range(2):
        p = [16, 32, 48, 64]
        p[3] = p[i]
        assert L.moe_grouped_mm(*ok, *p, None) == bad
        assert L.moe_grouped_mm_dx(*ok, *p, None) == bad
        assert L.moe_grouped_mm_dw(*ok, *p, 0, 0, None) == bad
    for flags in [(2, 0), (0, 2), (-1, 0), (1, 1)]:
        assert L.moe_grouped_mm_dw(*ok, 16, 32, 48, 64, *flags, None) == bad, flags
    # nothing to do
    assert L.moe_grouped_mm(4, 0, 64, 128, None, None, None, None, None) == moe.OK
    assert L.moe_grouped_mm_dw(4, 0, 64, 128, None, None, 48, 64, 0, 1, None) == moe.OK


def test_grouped_binding_refuses():
    import torch
    bf = dict(dtype=torch.bfloat16)
    x, w, y = torch.zeros(9, 16, **bf), torch.zeros(2, 24, 16, **bf), torch.zeros(9, 24, **bf)
    off = torch.zeros(3, dtype=torch.int32)
    for args, what in [((x, w, off, y[:8]), "must be"), ((x, w[0], off, y), "n_groups"),
                       ((x.float(), w, off, y), "float32"), ((x, w, off.long(), y), "int64"),
                       ((x, w, off[:2], y), "holds"), ((x, w, off, y.t()), "must be"),
                       ((x, w.transpose(1, 2), off, y), "must be|contiguous"),
                       ((x, w, off, y), "CUDA")]:
        with pytest.raises(moe.MoeError, match=what) as e:
            moe.moe_grouped_mm(*args)
        assert e.value.status == moe.ERR_INVALID_ARG
    with pytest.raises(moe.MoeError, match="CUDA"):
        moe.moe_grouped_mm_dx(y, w, off, x)
    with pytest.raises(moe.MoeError, match="float16"):
        moe.moe_grouped_mm_dw(y, x, off, w.half())


# ---------------------------------------------------------------- AdamW
def test_oracle_codes_and_random_words():
    import torch
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(block.e4m3_value(codes), want)
    np.testing.assert_array_equal(block.e4m3_position(want[:0x7f]), np.arange(0x7f))
    # the words are uniform and independent of one another: 2^16 of them, five standard deviations
    w = np.concatenate([block.random_words(1 << 14, t, s, k)
                        for t, s, k in ((0, 1, 1), (1, 1, 1), (0, 2, 1), (0, 1, 2))])
    assert len(np.unique(w)) > len(w) - 8
    for part in (w & 0xffff, w >> 16):
        z = part / 65536 - 0.5
        assert abs(z.mean()) < 5 / np.sqrt(12 * len(z))
        assert abs(np.mean(z[:-1] * z[1:])) < 5 / 12 / np.sqrt(len(z))


def adamw_entry(**kw):
    base = dict(p=1 << 20, grad=2 << 20, m=3 << 20, v=4 << 20, m_scale=5 << 20, v_scale=6 << 20,
                p_bf16=7 << 20, n=1000, weight_decay=0.1, grad_bf16=1)
    base.update(kw)
    return moe.MoeAdamwTensor(**base)


def make_table(entries, bits=8, short=0):
    L = moe.lib()
    array = (moe.MoeAdamwTensor * max(1, len(entries)))(*entries)
    size = L.moe_adamw_table_size(array, len(entries))
    if size == 0:
        return moe.ERR_INVALID_ARG, None, None
    image = ctypes.create_string_buffer(size)
    chunks = ctypes.c_int64(-1)
    rc = L.moe_adamw_table(array, len(entries), bits, image, size - short, ctypes.byref(chunks))
    return rc, chunks.value, image


def test_adamw_table():
    assert ctypes.sizeof(moe.MoeAdamwDesc) == 48 and ctypes.sizeof(moe.MoeAdamwTensor) == 72
    rc, chunks, _ = make_table([adamw_entry()])
    assert rc == moe.OK and chunks == 1
    rc, chunks, _ = make_table([])
    assert rc == moe.OK and chunks == 0
    far = {k: v + (64 << 20) for k, v in
           dict(p=1 << 20, grad=2 << 20, m=3 << 20, v=4 << 20, m_scale=5 << 20, v_scale=6 << 20,
                p_bf16=7 << 20).items()}
    rc, chunks, _ = make_table([adamw_entry(n=2048), adamw_entry(n=0, p=None),
                                adamw_entry(n=2049, **far)])
    assert rc == moe.OK and chunks == 3
    # two tensors may share a gradient, not what is written
    rc, chunks, _ = make_table([adamw_entry(), adamw_entry(**{**far, "grad": 2 << 20})])
    assert rc == moe.OK
    for k in ("p", "m", "v", "m_scale", "v_scale", "p_bf16"):
        kw = {**far, k: getattr(adamw_entry(), k)}
        assert make_table([adamw_entry(), adamw_entry(**kw)])[0] == moe.ERR_INVALID_ARG, k
        assert make_table([adamw_entry(grad=getattr(adamw_entry(), k))])[0] == moe.ERR_INVALID_ARG
    # the last element of one in the first of the next
    assert make_table([adamw_entry(), adamw_entry(**{**far, "p": (1 << 20) + 3996})])[0] != moe.OK
    assert make_table([adamw_entry(), adamw_entry(**{**far, "p": (1 << 20) + 4000})])[0] == moe.OK


@pytest.mark.parametrize("kw", [dict(p=None), dict(grad=None), dict(m=None), dict(v=None),
                                dict(m_scale=None), dict(v_scale=None), dict(n=-1),
                                dict(n=1 << 43), dict(grad_bf16=2), dict(p=(1 << 20) + 2),
                                dict(grad=(2 << 20) + 1), dict(p_bf16=(7 << 20) + 1),
                                dict(m_scale=(5 << 20) + 2),
                                dict(weight_decay=float("nan"))])
def test_adamw_table_refuses(kw):
    assert make_table([adamw_entry(**kw)])[0] == moe.ERR_INVALID_ARG
    if "scale" not in str(kw):
        assert make_table([adamw_entry(**kw)], bits=32)[0] == moe.ERR_INVALID_ARG


def test_adamw_refuses():
    L, bad = moe.lib(), moe.ERR_INVALID_ARG
    assert make_table([adamw_entry()], bits=16)[0] == bad
    assert make_table([adamw_entry()], short=1)[0] == moe.ERR_WORKSPACE
    d = moe.make_adamw_desc(1e-3)
    r = ctypes.byref(d)
    assert L.moe_adamw(r, None, 0, 0, 1, None, None, None) == moe.OK
    assert L.moe_adamw(None, 16, 1, 1, 1, None, None, None) == bad
    for args in [(16, 1, 1, 0, None, None), (16, 1, 1, -3, None, None), (None, 1, 1, 1, None, None),
                 (24, 1, 1, 1, None, None), (16, 0, 1, 1, None, None), (16, -1, 1, 1, None, None),
                 (16, 1, -1, 1, None, None), (16, 1, 1, 0, 2, None), (16, 1, 1, 1, None, 6),
                 (16, 1, 1 << 31, 1, None, None)]:
        assert L.moe_adamw(r, *args, None) == bad, args
    for kw in [dict(lr=float("nan")), dict(lr=float("inf")), dict(beta1=1.0), dict(beta1=-0.1),
               dict(beta2=1.0), dict(beta2=float("nan")), dict(eps=0.0), dict(eps=1e-60),
               dict(eps=float("inf")), dict(state_bits=16)]:
        x = moe.make_adamw_desc(**{"lr": 1e-3, **kw})
        assert L.moe_adamw(ctypes.byref(x), 16, 1, 1, 1, None, None, None) == bad, kw


def test_adamw_binding_refuses():
    import torch
    f = torch.zeros(256)
    e = torch.zeros(256, dtype=torch.uint8)
    s = torch.zeros(2)
    for kw, what in [(dict(grad=[f.double()]), "float64"), (dict(m=[e]), "uint8"),
                     (dict(v=[f[:200]]), "holds"), (dict(p=[f[::2]]), "contiguous"),
                     (dict(p_bf16=[f]), "float32"), (dict(m=[f, f]), "not a list"),
                     (dict(m_scale=[s]), "v_scale is not"), (dict(p=[None]), "missing"),
                     (dict(weight_decay=[0.1, 0.2]), "weight_decay is not"),
                     (dict(m_scale=[s], v_scale=[s]), "float32, not"),
                     (dict(m=[e], v=[e], m_scale=[s[:1]], v_scale=[s]), "holds"),
                     (dict(), "CUDA")]:
        with pytest.raises(moe.MoeError, match=what) as err:
            moe.adamw_table(**{**dict(p=[f], grad=[f], m=[f], v=[f]), **kw})
        assert err.value.status == moe.ERR_INVALID_ARG
    for step in (0, -1, 2 ** 31, 2 ** 32 + 1):
        with pytest.raises(moe.MoeError, match="step"):
            moe.moe_adamw(moe.make_adamw_desc(1e-3), moe.AdamwTable(None, 0, 0, 32, []), step)
    with pytest.raises(moe.MoeError, match="8-bit"):
        moe.moe_adamw(moe.make_adamw_desc(1e-3), moe.AdamwTable(None, 0, 0, 8, []), 1)
