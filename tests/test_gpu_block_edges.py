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
