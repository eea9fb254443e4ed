"""Accuracy of the grouped products over long contractions: the error is to stay that of fp32
addition, not to grow with every step of the tensor cores, which cut their sums off.

Tolerances.  Products of bf16 values are exact in fp32.  The contraction is taken in segments, of 512
rows for weight gradients and of 1024 else.  In a segment of length s a tensor-core step adds 16
products to the accumulator, each aligned to the largest of them and the sum rounded or cut once:
s / 16 + 17 units of 2^-23 of the segment's sum of magnitudes at most.  The n segments are added in
fp32, rounded to nearest: n more errors of 2^-24 of running sums, which stay below the whole sum of
magnitudes M.  In all ((s / 16 + 17) 2^-23 + n 2^-24) M; a bf16 output adds half a step, 2^-8 of its
value.  (Accumulated in one go, products of one sign would lose up to k / 16 units of 2^-23 of M: 33000
rows 2.5e-4 M instead of 9.7e-6 M.)
"""
import pytest
import torch

import forward_moe_route_b200 as moe

pytestmark = pytest.mark.gpu

BF = dict(dtype=torch.bfloat16, device="cuda")


def hold(name, got, want, magnitude, k, segment, half=0.0, start=0.0):
    off = (got.double() - want).abs()
    bound = (segment / 16 + 17) * 2.0 ** -23 + -(-k // segment) * 2.0 ** -24
    tol = bound * magnitude + half * want.abs() + 2.0 ** -24 * start
    assert bool((off <= tol).all()), f"{name}: {float((off / magnitude).max()):.2e} of M"


def draw(gen, kind, *shape):
    x = torch.randn(*shape, generator=gen, device="cuda")
    return (x.abs() if kind == "positive" else x).to(torch.bfloat16)


@pytest.mark.parametrize("kind", ["random", "positive"])
@pytest.mark.parametrize("loads", [[33000], [511, 512, 513, 0, 1024, 1025, 5000], [1537, 40001, 7]])
def test_weight_gradients_of_many_rows(loads, kind):
    gen = torch.Generator(device="cuda").manual_seed(len(loads))
    d_in, d_out = 264, 312
    x, dy = draw(gen, kind, sum(loads), d_in), draw(gen, kind, sum(loads), d_out)
    offsets = torch.tensor([0] + torch.tensor(loads).cumsum(0).tolist(), dtype=torch.int32,
                           device="cuda")
    G = len(loads)
    dw = torch.full((G, d_out, d_in), float("nan"), device="cuda")
    db = torch.full((G, d_out, d_in), float("nan"), **BF)
    start = torch.randn(G, d_out, d_in, generator=gen, device="cuda")
    acc = start.clone()
    moe.moe_grouped_mm_dw(dy, x, offsets, dw)
    moe.moe_grouped_mm_dw(dy, x, offsets, db)
    moe.moe_grouped_mm_dw(dy, x, offsets, acc, accumulate=True)
    assert moe.moe_last_device_status() == moe.OK
    at = 0
    for g, n in enumerate(loads):
        a, b = dy[at:at + n].double(), x[at:at + n].double()
        at += n
        want, size = a.T @ b, a.abs().T @ b.abs()
        if n == 0:
            assert (dw[g] == 0).all() and (db[g] == 0).all() and torch.equal(acc[g], start[g])
            continue
        hold("dw", dw[g], want, size, n, 512)
        hold("dw bf16", db[g], want, size, n, 512, half=2.0 ** -8)
        first = start[g].double()
        hold("dw +=", acc[g], first + want, size, n, 512, start=first.abs() + size)


# outputs near zero beside running sums that are not: the second half of the contraction takes back
# what the first half adds up, so what is left shows the error of the sums and little rounding
@pytest.mark.parametrize("rows", [[40], [300, 0, 5, 1], [3, 1]])
@pytest.mark.parametrize("k", [520, 1024, 7168, 32768])
def test_long_products(k, rows):
    gen = torch.Generator(device="cuda").manual_seed(k)
    R, G, f = sum(rows), len(rows), 136
    x, w = draw(gen, "positive", R, k), draw(gen, "positive", G, f, k)
    x[:, k // 2:] = -x[:, :k // 2]
    w[:, :, k // 2:] = w[:, :, :k // 2]
    w[:, :, ::97] += 0.5
    offsets = torch.tensor([0] + torch.tensor(rows).cumsum(0).tolist(), dtype=torch.int32,
                           device="cuda")
    y, dx = torch.empty(R, f, **BF), torch.empty(R, f, **BF)
    moe.moe_grouped_mm(x, w, offsets, y)
    moe.moe_grouped_mm_dx(x, w.transpose(1, 2).contiguous(), offsets, dx)
    assert moe.moe_last_device_status() == moe.OK
    at = 0
    for g, n in enumerate(rows):
        a, b = x[at:at + n].double(), w[g].double().T
        want, size = a @ b, a.abs() @ b.abs()
        hold("y", y[at:at + n], want, size, k, 1024, half=2.0 ** -8) if n else None
        hold("dx", dx[at:at + n], want, size, k, 1024, half=2.0 ** -8) if n else None
        at += n
