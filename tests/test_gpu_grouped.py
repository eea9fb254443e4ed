"""GPU parity of the grouped products (moe_grouped_mm, _dx, _dw) with the fp64 oracle.

Tolerances, from the arithmetic.  Products of bf16 values are exact in fp32.  A contraction of
length k is k / 16 tensor-core steps; a step adds 16 products to the fp32 accumulator, each
aligned to the largest of them and the sum rounded or cut once, so at most 17 units of 2^-23 of the
sum of magnitudes M for the alignment and one unit of the running sum per step.  Running sums stay
below M: (k / 16 + 17) 2^-23 M in all.  A bf16 output adds half a step, 2^-8 of its value; adding to
dw in fp32 adds 2^-24 of the sum.
"""
import numpy as np
import pytest
import torch

import forward_moe_route_b200 as moe
from oracle import block

pytestmark = pytest.mark.gpu

BF = dict(dtype=torch.bfloat16, device="cuda")


def rand(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen) * std).to(torch.bfloat16).cuda()


def f64(t):
    return t.double().cpu().numpy()


def close(name, got, want, magnitude, k, bf16=True):
    got = f64(got)
    tol = (np.asarray(k) / 16 + 17) * 2.0 ** -23 * magnitude
    tol = tol + (2.0 ** -8 if bf16 else 2.0 ** -24) * np.abs(want)
    off = np.abs(got - want) - tol
    assert got.shape == want.shape and np.isfinite(got).all(), name
    assert (off <= 1e-30).all(), f"{name}: over by {off.max():.3e} at {np.argmax(off)}"


def offsets_of(loads, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(loads)]), dtype=torch.int32,
                        device="cuda")


def check(gen, loads, d_in, d_out, before=0, behind=0):
    """All three products of one ragged row list; rows of no group are NaN in the inputs."""
    G, R = len(loads), sum(loads) + before + behind
    off = offsets_of(loads, before)
    o = off.cpu().numpy()
    x, dy = rand(gen, R, d_in), rand(gen, R, d_out)
    outside = torch.ones(R, dtype=torch.bool, device="cuda")
    outside[before:R - behind] = False
    x[outside] = float("nan")
    dy[outside] = float("nan")
    w = rand(gen, G, d_out, d_in, std=0.1)
    X, DY, W = np.nan_to_num(f64(x)), np.nan_to_num(f64(dy)), f64(w)
    inside = ~outside.cpu().numpy()

    y = torch.full((R, d_out), 5.0, **BF)
    moe.moe_grouped_mm(x, w, off, y)
    close("y", y[~outside], block.grouped_mm(X, W, o, np.zeros((R, d_out)))[inside],
          block.grouped_mm(abs(X), abs(W), o, np.zeros((R, d_out)))[inside], d_in)
    assert (y[outside] == 5).all()
    dx = torch.full((R, d_in), 5.0, **BF)
    moe.moe_grouped_mm_dx(dy, w, off, dx)
    close("dx", dx[~outside], block.grouped_mm_dx(DY, W, o, np.zeros((R, d_in)))[inside],
          block.grouped_mm_dx(abs(DY), abs(W), o, np.zeros((R, d_in)))[inside], d_out)
    assert (dx[outside] == 5).all()

    zero = np.zeros((G, d_out, d_in))
    want, mag = block.grouped_mm_dw(DY, X, o, zero), block.grouped_mm_dw(abs(DY), abs(X), o, zero)
    k = np.array(loads).reshape(G, 1, 1)
    dw = torch.full((G, d_out, d_in), float("nan"), device="cuda")
    moe.moe_grouped_mm_dw(dy, x, off, dw)
    close("dw", dw, want, mag, k, bf16=False)
    db = torch.full((G, d_out, d_in), float("nan"), **BF)
    moe.moe_grouped_mm_dw(dy, x, off, db)
    close("dw bf16", db, want, mag, k)
    start = torch.randn(G, d_out, d_in, generator=gen).cuda()
    acc = start.clone()
    moe.moe_grouped_mm_dw(dy, x, off, acc, accumulate=True)
    close("dw +=", acc, want + f64(start), mag, k, bf16=False)
    empty = torch.tensor(loads, device="cuda") == 0
    assert torch.equal(acc[empty], start[empty])
    assert (dw[empty] == 0).all() and (db[empty] == 0).all()
    assert moe.moe_last_device_status() == moe.OK


# one-row groups, empty ones, ends inside and at the edges of the 16-, 32-, 64- and 256-row tiles
LOADS = [[1], [0, 1, 0], [16, 15, 17, 0, 33], [63, 64, 65, 1], [256, 255, 257, 0, 0, 31],
         [513, 2, 700], [1] * 70, [0] * 5 + [130]]


@pytest.mark.parametrize("loads", LOADS, ids=lambda v: f"{len(v)}g{sum(v)}")
@pytest.mark.parametrize("d_in,d_out", [(8, 8), (64, 256), (72, 264), (520, 136), (256, 1000)])
def test_products(loads, d_in, d_out):
    gen = torch.Generator().manual_seed(sum(loads) * 7 + d_in + d_out)
    check(gen, loads, d_in, d_out, before=3, behind=len(loads) % 3 * 9)


@pytest.mark.parametrize("G,d_in,d_out", [(1024, 64, 72), (300, 136, 64), (2, 2048, 4096)])
def test_many_groups_and_long_contractions(G, d_in, d_out):
    gen = torch.Generator().manual_seed(G)
    loads = torch.randint(0, 7 if G > 2 else 900, (G,), generator=gen).tolist()
    check(gen, loads, d_in, d_out)


def test_a_groups_nan_stays_in_it():
    gen = torch.Generator().manual_seed(5)
    loads = [20, 13, 0, 50, 3]
    off = offsets_of(loads)
    o = off.tolist()
    x, dy, w = rand(gen, 86, 264), rand(gen, 86, 136), rand(gen, 5, 136, 264)
    x[o[1]:o[2]] = float("nan")
    dy[o[3]:o[4]] = float("inf")
    y, dx = torch.empty(86, 136, **BF), torch.empty(86, 264, **BF)
    dw = torch.empty(5, 136, 264, device="cuda")
    moe.moe_grouped_mm(x, w, off, y)
    moe.moe_grouped_mm_dx(dy, w, off, dx)
    moe.moe_grouped_mm_dw(dy, x, off, dw)
    assert y[o[1]:o[2]].isnan().all() and y[:o[1]].isfinite().all() and y[o[2]:].isfinite().all()
    assert not dx[o[3]:o[4]].isfinite().any()
    assert dx[:o[3]].isfinite().all() and dx[o[4]:].isfinite().all()
    assert dw[1].isnan().all() and not dw[3].isfinite().any() and dw[[0, 2, 4]].isfinite().all()
    assert moe.moe_last_device_status() == moe.OK


@pytest.mark.parametrize("offsets", [[0, 20, 10, 30], [-4, 10, 20, 30], [0, 10, 20, 41],
                                     [50, 60, 70, 80]])
def test_offsets_out_of_order_are_reported_and_read_as_empty(offsets):
    gen = torch.Generator().manual_seed(6)
    x, w = rand(gen, 40, 64), rand(gen, 3, 72, 64)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    y = torch.full((40, 72), 5.0, **BF)
    dw = torch.full((3, 72, 64), float("nan"), device="cuda")
    moe.moe_grouped_mm(x, w, off, y)
    assert moe.moe_last_device_status() == moe.ERR_DEVICE_CHECK
    moe.moe_grouped_mm_dw(y, x, off, dw)
    assert moe.moe_last_device_status() == moe.ERR_DEVICE_CHECK
    for g, (a, b) in enumerate(zip(offsets[:-1], offsets[1:])):
        if not 0 <= a <= b <= 40:
            assert (dw[g] == 0).all()
    held = {r for a, b in zip(offsets[:-1], offsets[1:]) if 0 <= a <= b <= 40
            for r in range(a, b)}
    for r in range(40):
        assert r in held or (y[r] == 5).all()


def test_no_rows():
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    x, y = torch.empty(0, 64, **BF), torch.empty(0, 72, **BF)
    w = torch.ones(2, 72, 64, **BF)
    moe.moe_grouped_mm(x, w, off, y)
    moe.moe_grouped_mm_dx(y, w, off, x)
    for dw in (torch.full((2, 72, 64), 3.0, device="cuda"), torch.full((2, 72, 64), 3.0, **BF)):
        moe.moe_grouped_mm_dw(y, x, off, dw)
        assert (dw == 0).all()
    keep = torch.full((2, 72, 64), 3.0, device="cuda")
    moe.moe_grouped_mm_dw(y, x, off, keep, accumulate=True)
    assert (keep == 3).all()


def test_graph_follows_the_offsets_and_two_runs_agree():
    gen = torch.Generator().manual_seed(9)
    x, dy, w = rand(gen, 700, 264), rand(gen, 700, 136), rand(gen, 6, 136, 264)
    a, b = offsets_of([100, 0, 300, 17, 200, 83]), offsets_of([1, 650, 0, 0, 9, 40])
    off = a.clone()

    def outputs():
        return (torch.zeros(700, 136, **BF), torch.zeros(700, 264, **BF),
                torch.zeros(6, 136, 264, device="cuda"))

    def passes(o, y, dx, dw):
        moe.moe_grouped_mm(x, w, o, y)
        moe.moe_grouped_mm_dx(dy, w, o, dx)
        moe.moe_grouped_mm_dw(dy, x, o, dw)

    held = outputs()
    passes(off, *held)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        passes(off, *held)
    for o in (b, a):
        off.copy_(o)
        graph.replay()
        eager = outputs()
        passes(o, *eager)
        for p, q in zip(held, eager):
            assert torch.equal(p, q)
    assert moe.moe_last_device_status() == moe.OK


# a handful of rows: alone, in one group, in more than a pass of a group holds, with gaps
@pytest.mark.parametrize("loads", [[1], [16], [5, 0, 2], [0, 0, 3, 4, 9], [1] * 9, [0] * 40 + [7]],
                         ids=lambda v: f"{len(v)}g{sum(v)}")
@pytest.mark.parametrize("d_in,d_out", [(8, 16), (64, 72), (1000, 264), (2048, 24), (40, 2056)])
def test_a_handful_of_rows(loads, d_in, d_out):
    gen = torch.Generator().manual_seed(sum(loads) + d_in + d_out)
    check(gen, loads, d_in, d_out)
    if sum(loads) < 14:
        check(gen, loads, d_in, d_out, before=1, behind=1)
