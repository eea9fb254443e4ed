"""Edges of the operators around the layer on the GPU."""
import pytest
import torch

import forward_moe_route_b200 as moe

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate_group", [0, 1, 4, 1 << 20])
def test_no_tokens_through_the_end_of_a_block(gate_group, dtype):
    d, slots = 256, 3
    desc = moe.make_norm_desc(0, d, EPS, "f32" if dtype == torch.float32 else "bf16", slots,
                              gate_group)
    like = dict(dtype=dtype, device="cuda")
    rows, w = torch.empty(0, d, **like), torch.ones(d, **like)
    gate = torch.empty(0, d, **like) if gate_group else None
    ys = torch.empty(0, slots, d, **like)
    moe.moe_combine_norm(desc, rows, ys, w, gate, None, rows, None, None)
    moe.moe_combine_norm(desc, rows, ys, w, gate, w, rows, rows, rows)
    dw = torch.full((d,), 7.0, device="cuda")
    ws = moe.norm_backward_workspace(desc)
    moe.moe_combine_norm_backward(desc, rows, w, gate, rows, rows, dw, gate, ws)
    assert (dw == 0).all()
    dw.fill_(7.0)
    moe.moe_norm_backward(desc, rows, w, rows, None, rows, dw, ws)
    assert (dw == 0).all()
    assert moe.moe_last_device_status() == moe.OK


def test_weight_gradients_follow_offsets_that_the_kernel_before_wrote():
    """Routing, permutation and weight gradients back to back, the loads of the experts different
    each time; then the same products from copies of the offsets, one at a time."""
    T, D, INNER, N, K, PASSES = 333, 256, 136, 8, 2, 24
    gen = torch.Generator().manual_seed(11)

    def draw(*shape):
        return torch.randn(*shape, generator=gen).to(torch.bfloat16).cuda()

    layer = moe.make_desc(T, D, 0, N, K, 128, "sigmoid", True, 1.0)
    ws = moe.workspace(layer)
    xs, router, dy = [draw(T, D) for _ in range(PASSES)], draw(N, D), draw(T * K, INNER)
    i32 = dict(dtype=torch.int32, device="cuda")
    idx, counts, offsets = torch.empty(T, K, **i32), torch.empty(N, **i32), torch.empty(N + 1, **i32)
    src, slot = torch.empty(T * K, **i32), torch.empty(T * K, **i32)
    weight = torch.empty(T, K, device="cuda")
    x_perm = torch.empty(T * K, D, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    kept = []
    for x in xs:
        dw = torch.full((N, INNER, D), float("nan"), device="cuda")
        moe.moe_route(layer, x, router, None, idx, weight, counts, ws)
        moe.moe_permute(layer, x, idx, counts, offsets, src, slot, x_perm, None, ws)
        moe.moe_grouped_mm_dw(dy, x_perm, offsets, dw)
        kept.append((dw, offsets.clone(), x_perm.clone()))
    assert moe.moe_last_device_status() == moe.OK
    assert len({tuple(o.tolist()) for _, o, _ in kept}) > PASSES // 2
    for dw, o, rows in kept:
        again = torch.empty_like(dw)
        torch.cuda.synchronize()
        moe.moe_grouped_mm_dw(dy, rows, o, again)
        assert torch.equal(dw, again)
