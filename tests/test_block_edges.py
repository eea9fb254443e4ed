"""Edges of the operators around the layer that need no GPU: batches without tokens."""
import ctypes

import pytest

import forward_moe_route_b200 as moe


# An empty tensor's address is null, so without tokens every array that holds rows may be null:
# [T, ...] and the gate's ceil(T / gate_group) rows.  The weights [d] are there all the same.
@pytest.mark.parametrize("gate_group", [0, 1, 4, 1 << 20])
def test_no_tokens_and_null_addresses(gate_group):
    L = moe.lib()
    d = moe.make_norm_desc(0, 256, 1e-6, n_slots=2, gate_group=gate_group)
    r, w, w_next, dw, ws = ctypes.byref(d), 32, 48, 64, 80
    small = moe.moe_norm_backward_workspace_size(d) - 1
    for gate in (None, 96) if gate_group else (None,):
        for follow in (None, w_next):
            assert L.moe_combine_norm(r, None, None, w, gate, follow, None, None, None,
                                      None) == moe.OK
        # past the checks of the arguments: the first thing that is refused is the workspace
        assert L.moe_combine_norm_backward(r, None, w, gate, None, None, dw, None, ws, small,
                                           None) == moe.ERR_WORKSPACE
        assert L.moe_norm_backward(r, None, w, None, None, None, dw, ws, small,
                                   None) == moe.ERR_WORKSPACE
    assert L.moe_norm(r, None, w, None, None) == moe.OK


def test_no_tokens_do_not_excuse_other_mistakes():
    L, bad = moe.lib(), moe.ERR_INVALID_ARG
    plain, gated = (moe.make_norm_desc(0, 256, 1e-6, gate_group=g) for g in (0, 4))
    p, g = ctypes.byref(plain), ctypes.byref(gated)
    # a gate, or its gradient, without gate_group; x_next without w_next; no place for dw
    assert L.moe_combine_norm(p, None, None, 32, 48, None, None, None, None, None) == bad
    assert L.moe_combine_norm(g, None, None, 32, None, None, None, None, 48, None) == bad
    assert L.moe_combine_norm_backward(p, None, 32, 48, None, None, 64, None, 80, 0, None) == bad
    assert L.moe_combine_norm_backward(p, None, 32, None, None, None, 64, 48, 80, 0, None) == bad
    assert L.moe_combine_norm_backward(g, None, 32, None, None, None, None, None, 80, 0,
                                       None) == bad
    # and with tokens they are needed
    one = moe.make_norm_desc(1, 256, 1e-6, gate_group=4)
    o = ctypes.byref(one)
    assert L.moe_combine_norm(o, 16, 32, 48, None, None, 64, None, None, None) == bad
    assert L.moe_combine_norm(o, 16, 32, 48, 80, 96, 64, None, None, None) == bad
    assert L.moe_combine_norm_backward(o, 16, 32, 48, 64, 80, 96, None, 112, 0, None) == bad


def test_adamw_takes_the_rate_and_the_step_on_the_device_as_tensors():
    """A number for lr would be read as an address, 0 as no rate at all."""
    table = moe.AdamwTable(None, 0, 0, 32, [])
    desc = moe.make_adamw_desc(1e-3)
    for lr in (0, 0.0, 1e-3, 16):
        with pytest.raises(moe.MoeError, match="lr") as e:
            moe.moe_adamw(desc, table, 1, lr=lr)
        assert e.value.status == moe.ERR_INVALID_ARG
    for step in (2.0, None, "3"):
        with pytest.raises(moe.MoeError, match="step") as e:
            moe.moe_adamw(desc, table, step)
        assert e.value.status == moe.ERR_INVALID_ARG


def test_grouped_products_name_what_is_missing():
    import torch
    bf = dict(dtype=torch.bfloat16)
    x, w, y = torch.zeros(9, 16, **bf), torch.zeros(2, 24, 16, **bf), torch.zeros(9, 24, **bf)
    off = torch.zeros(3, dtype=torch.int32)
    for call, args, names in ((moe.moe_grouped_mm, (x, w, off, y), "x w offsets y"),
                              (moe.moe_grouped_mm_dx, (y, w, off, x), "dy w offsets dx"),
                              (moe.moe_grouped_mm_dw, (y, x, off, w), "dy x offsets dw")):
        for i, name in enumerate(names.split()):
            with pytest.raises(moe.MoeError, match=f"{name} is missing") as e:
                call(*args[:i], None, *args[i + 1:])
            assert e.value.status == moe.ERR_INVALID_ARG
