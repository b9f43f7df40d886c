"""The gated route, the gradients and the 4-bit products refuse what they cannot do, on the host, before anything is
launched (no GPU needed)."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def moe():
    from combine_router_top_gb300 import build as B
    B.build()
    import combine_router_top_gb300 as M
    return M


FAKE, ODD = C.c_void_p(1 << 40), C.c_void_p((1 << 40) + 2)


def route(M, p, g, logits=FAKE, bias=FAKE, outs=None, ws=FAKE, n=1 << 24):
    return M.lib().moe_route_gated(C.byref(p) if p else None, C.byref(g) if g else None, logits, bias,
                                   *(outs or [FAKE] * 7), ws, n, None)


@pytest.mark.parametrize("bad", [
    dict(score=2), dict(score=-1), dict(groups=0), dict(groups=7), dict(groups=8, top_groups=0),
    dict(groups=8, top_groups=9), dict(group_rule=2), dict(logits_type=2), dict(scale=0.0),
    dict(scale=float("inf")), dict(scale=float("nan")), dict(groups=64, top_groups=1),
    dict(groups=256, top_groups=8, group_rule=1)])
def test_gates(moe, bad):
    p = moe.problem(100, 8, 256, 8, 8, 128)
    g = moe.gate(**bad)
    assert route(moe, p, g) == moe.MOE_ERR_INVALID_ARG
    assert moe.lib().moe_route_gated_backward(C.byref(p), C.byref(g), FAKE, FAKE, FAKE, FAKE, FAKE,
                                              None) == moe.MOE_ERR_INVALID_ARG


def test_more_groups_than_lanes_are_unsupported(moe):
    p = moe.problem(100, 8, 256, 8, 8, 128)
    assert route(moe, p, moe.gate(groups=64)) == moe.MOE_ERR_UNSUPPORTED


def test_route_buffers(moe):
    p, g = moe.problem(100, 8, 256, 8, 8, 128), moe.gate(groups=8, top_groups=4)
    assert route(moe, None, g) == route(moe, p, None) == moe.MOE_ERR_INVALID_ARG
    assert route(moe, moe.problem(100, 8, 256, 17, 8, 128), g) == moe.MOE_ERR_INVALID_ARG
    assert route(moe, p, g, logits=None) == route(moe, p, g, logits=ODD) == moe.MOE_ERR_INVALID_ARG
    assert route(moe, p, g, bias=ODD) == route(moe, p, g, ws=None) == moe.MOE_ERR_INVALID_ARG
    assert route(moe, p, g, n=moe.moe_route_workspace_bytes(p) - 1) == moe.MOE_ERR_INVALID_ARG
    for i in range(7):
        for b in (None, ODD):
            outs = [FAKE] * 7
            outs[i] = b
            assert route(moe, p, g, outs=outs) == moe.MOE_ERR_INVALID_ARG, i
    # rows of 16-byte multiples need 16-byte alignment, others the element's
    eight = C.c_void_p((1 << 40) + 8)
    assert route(moe, p, g, logits=eight) == moe.MOE_ERR_INVALID_ARG
    assert route(moe, p, moe.gate(logits_type=moe.MOE_LOGITS_BF16), logits=eight) == moe.MOE_ERR_INVALID_ARG


def test_route_backward_buffers(moe):
    f = moe.lib().moe_route_gated_backward
    p = moe.problem(100, 8, 256, 8, 8, 128)
    dense, sig, sm = moe.gate(renormalise=False), moe.gate(moe.MOE_SCORE_SIGMOID), moe.gate()
    for g in (dense, sig):
        assert f(C.byref(p), C.byref(g), None, FAKE, FAKE, FAKE, FAKE, None) == moe.MOE_ERR_INVALID_ARG
    assert f(None, C.byref(sm), FAKE, FAKE, FAKE, FAKE, FAKE, None) == moe.MOE_ERR_INVALID_ARG
    for i in range(4):
        for b in (None, ODD):
            a = [FAKE] * 4
            a[i] = b
            assert f(C.byref(p), C.byref(sm), FAKE, *a, None) == moe.MOE_ERR_INVALID_ARG
    assert f(C.byref(moe.problem(0, 8, 256, 8, 8, 128)), C.byref(sm), None, None, None, None, None, None) == moe.MOE_OK


def test_combine_backward_buffers(moe):
    f = moe.lib().moe_combine_backward
    p = moe.problem(100, 64, 16, 4, 4, 32)
    for i in range(7):
        for b in (None, ODD):
            a = [FAKE] * 7
            a[i] = b
            assert f(C.byref(p), *a, None) == moe.MOE_ERR_INVALID_ARG, i
    assert f(None, *[FAKE] * 7, None) == moe.MOE_ERR_INVALID_ARG
    assert f(C.byref(moe.problem(0, 64, 16, 4, 4, 32)), *[None] * 7, None) == moe.MOE_OK


@pytest.mark.parametrize("bad", [dict(n_in=64), dict(n_in=192), dict(n_in=0), dict(n_in=65536 + 128), dict(n_out=4),
                                 dict(n_out=12), dict(n_out=0), dict(n_out=65544), dict(group=16), dict(group=256),
                                 dict(group=0), dict(act=2), dict(act=-1)])
def test_w4_shapes(moe, bad):
    p = moe.problem(100, 64, 16, 4, 4, 32)
    w = moe.w4(**{**dict(n_in=256, n_out=64, group=64, act=0), **bad})
    assert moe.moe_expert_w4_workspace_bytes(p, w) == 0
    assert moe.lib().moe_expert_w4(C.byref(p), C.byref(w), FAKE, None, *[FAKE] * 5, 1 << 30,
                                   None) == moe.MOE_ERR_INVALID_ARG


def test_w4_buffers(moe):
    f = moe.lib().moe_expert_w4
    pb, pf, w = moe.problem(100, 64, 16, 4, 4, 32), moe.problem(100, 128, 16, 4, 4, 32, 1), moe.w4(256, 64, 64)
    n = moe.moe_expert_w4_workspace_bytes(pb, w)
    assert n > 0 and moe.moe_expert_w4_workspace_bytes(pf, w) > 0
    # scales exactly for fp8 rows
    assert f(C.byref(pb), C.byref(w), FAKE, FAKE, *[FAKE] * 5, 1 << 40, None) == moe.MOE_ERR_INVALID_ARG
    assert f(C.byref(pf), C.byref(w), FAKE, None, *[FAKE] * 5, 1 << 40, None) == moe.MOE_ERR_INVALID_ARG
    assert f(C.byref(pf), C.byref(w), FAKE, ODD, *[FAKE] * 5, 1 << 40, None) == moe.MOE_ERR_INVALID_ARG
    assert f(C.byref(pb), C.byref(w), FAKE, None, *[FAKE] * 5, n - 1, None) == moe.MOE_ERR_INVALID_ARG
    assert f(None, C.byref(w), FAKE, None, *[FAKE] * 5, n, None) == moe.MOE_ERR_INVALID_ARG
    assert f(C.byref(pb), None, FAKE, None, *[FAKE] * 5, n, None) == moe.MOE_ERR_INVALID_ARG
    for i in range(6):                                  # x, counts, w_q, w_scale, y, workspace
        for b in (None, ODD):
            a = [FAKE] * 6
            a[i] = b
            assert f(C.byref(pb), C.byref(w), a[0], None, *a[1:], 1 << 40, None) == moe.MOE_ERR_INVALID_ARG, i
    p0 = moe.problem(0, 64, 16, 4, 4, 32)
    assert f(C.byref(p0), C.byref(w), None, None, *[None] * 5, 0, None) == moe.MOE_OK


def test_the_binding_takes_cuda_tensors_and_whole_blocks(moe):
    import torch
    t = torch.zeros(16, dtype=torch.int32)
    p = moe.problem(4, 256, 8, 2, 2, 4)
    with pytest.raises(ValueError):
        moe.moe_combine_backward(p, t, t, t, t, t, t, t)
    with pytest.raises(ValueError):
        moe.w4_pack(torch.zeros((4, 120), dtype=torch.uint8))
    with pytest.raises(ValueError):
        moe.w4_pack(torch.zeros((4, 128), dtype=torch.int32))
