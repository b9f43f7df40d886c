"""The norms around a block and the layer for a few tokens refuse what they cannot do, on the host, before anything is
launched (no GPU needed)."""
import ctypes as C

import pytest

FAKE, ODD = C.c_void_p(1 << 40), C.c_void_p((1 << 40) + 2)
INF = float("inf")


@pytest.fixture(scope="module")
def M():
    from combine_router_top_gb300 import build as B
    B.build()
    import combine_router_top_gb300 as M
    return M


def block(M, p, n, y=FAKE, residual=FAKE, post=FAKE, pre=FAKE, gate=None, r=FAKE, out=FAKE):
    return M.lib().moe_block_norm(C.byref(p) if p else None, C.byref(n) if n else None, y, residual, post, pre, gate, r, out,
                                  None)


def combine(M, p, n, y=FAKE, idx=FAKE, w=FAKE, slot=FAKE, residual=FAKE, post=FAKE, pre=FAKE, gate=None, keep=None, r=FAKE,
            out=FAKE):
    return M.lib().moe_combine_norm(C.byref(p), C.byref(n), y, idx, w, slot, residual, post, pre, gate, keep, r, out, None)


def back(M, p, n, y=FAKE, r=FAKE, d_r=FAKE, d_n=FAKE, post=FAKE, pre=FAKE, gate=None, d_y=FAKE, d_res=FAKE, d_post=None,
         d_pre=None, d_gate=None, ws=FAKE, size=1 << 40):
    return M.lib().moe_block_norm_backward(C.byref(p), C.byref(n), y, r, d_r, d_n, post, pre, gate, d_y, d_res, d_post, d_pre,
                                           d_gate, ws, size, None)


@pytest.mark.parametrize("bad", [dict(eps=0.0), dict(eps=-1e-6), dict(eps=INF), dict(eps=float("nan")), dict(scale=INF),
                                 dict(scale=float("nan")), dict(gate=3), dict(gate=-1), dict(residual=2), dict(params=2)])
def test_norms(M, bad):
    p, n = M.problem(4, 64, 8, 2, 1, 4), M.norm(**bad)
    gate = FAKE if bad.get("gate") else None
    assert block(M, p, n, gate=gate) == combine(M, p, n, gate=gate) == back(M, p, n, gate=gate) == M.MOE_ERR_INVALID_ARG
    assert M.moe_block_norm_backward_workspace_bytes(p, n) == 0


def test_wide_rows_are_unsupported(M):
    p, n = M.problem(4, 16392, 8, 2, 1, 4), M.norm()
    assert block(M, p, n) == combine(M, p, n) == back(M, p, n) == M.MOE_ERR_UNSUPPORTED
    assert M.moe_block_norm_backward_workspace_bytes(p, n) == 0
    assert M.moe_block_norm_backward_workspace_bytes(M.problem(4, 16384, 8, 2, 1, 4), n) > 0


def test_block_norm_buffers(M):
    p, n, bad = M.problem(4, 64, 8, 2, 1, 4), M.norm(), M.MOE_ERR_INVALID_ARG
    assert block(M, None, n) == block(M, p, None) == block(M, M.problem(4, 65, 8, 2, 1, 4), n) == bad
    for k in ("y", "residual", "post", "pre", "r", "out"):
        assert block(M, p, n, **{k: ODD}) == bad, k
    assert block(M, p, n, residual=None) == block(M, p, n, r=None, out=None, pre=None) == bad
    assert block(M, p, n, pre=None) == block(M, p, n, out=None) == bad                  # n exactly with its weights
    assert block(M, p, n, gate=FAKE) == bad                                             # a gate that norm does not name
    for kind in (M.MOE_BRANCH_CHANNEL, M.MOE_BRANCH_TOKEN):
        assert block(M, p, M.norm(gate=kind)) == block(M, p, M.norm(gate=kind), gate=ODD) == bad
    # no block: the residual alone, no r, no weights after a block
    assert block(M, p, n, y=None, post=None) == block(M, p, n, y=None, r=None) == bad
    assert block(M, p, M.norm(gate=1), y=None, post=None, gate=FAKE, r=None) == bad
    assert block(M, M.problem(0, 64, 8, 2, 1, 4), n, *[None] * 7) == M.MOE_OK


def test_combine_norm_buffers(M):
    p, n = M.problem(4, 64, 8, 2, 1, 4), M.norm()
    for k in ("y", "idx", "w", "slot", "residual"):
        for b in (None, ODD):
            assert combine(M, p, n, **{k: b}) == M.MOE_ERR_INVALID_ARG, k
    for k in ("post", "pre", "keep", "r", "out"):
        assert combine(M, p, n, **{k: ODD}) == M.MOE_ERR_INVALID_ARG, k
    assert combine(M, M.problem(0, 64, 8, 2, 1, 4), n, *[None] * 11) == M.MOE_OK


def test_backward_buffers(M):
    p, n, bad = M.problem(4, 64, 8, 2, 1, 4), M.norm(), M.MOE_ERR_INVALID_ARG
    for k in ("y", "r", "d_r", "d_n", "post", "pre", "d_y", "d_res", "d_post", "d_pre", "ws"):
        assert back(M, p, n, **{k: ODD}) == bad, k
    for k in ("r", "d_n", "d_y", "d_res", "ws"):
        assert back(M, p, n, **{k: None}) == bad, k
    assert back(M, p, n, size=M.moe_block_norm_backward_workspace_bytes(p, n) - 1) == bad
    assert back(M, p, n, d_r=None, d_n=None, pre=None) == bad                           # no gradient comes in
    assert back(M, p, n, gate=FAKE) == back(M, p, n, d_gate=FAKE) == bad
    assert back(M, p, n, post=None, d_post=FAKE) == back(M, p, n, pre=None, d_n=None, d_pre=FAKE) == bad
    assert back(M, p, n, y=None) == back(M, p, n, y=None, d_y=None) == bad              # weights after no block
    assert back(M, M.problem(0, 64, 8, 2, 1, 4), n, *[None] * 11) == M.MOE_OK


def few(M, p, g, m, x=FAKE, logits=FAKE, bias=None, up=FAKE, us=None, down=FAKE, ds=None, idx=None, w=None, out=FAKE, ws=FAKE,
        size=1 << 40):
    return M.lib().moe_layer_few(C.byref(p) if p else None, C.byref(g) if g else None, C.byref(m) if m else None, x, logits,
                                 bias, up, us, down, ds, idx, w, out, ws, size, None)


@pytest.mark.parametrize("bad", [dict(inner=0), dict(inner=65600), dict(weights=3), dict(weights=-1), dict(shared=2),
                                 dict(shared=-1), dict(weights=2, group=16), dict(weights=2, group=0)])
def test_mlps(M, bad):
    p, m = M.problem(4, 256, 8, 2, 1, 4), M.mlp(**{**dict(inner=256), **bad})
    scale = FAKE if bad.get("weights") else None
    assert few(M, p, M.gate(), m, us=scale, ds=scale) == M.MOE_ERR_INVALID_ARG
    assert M.moe_layer_few_workspace_bytes(p, m) == 0


def test_what_the_few_kernels_do_not_take(M):
    ok = dict(T=4, H=256, E=8, k=2, R=1, Cap=4)
    for change, m in [(dict(T=33), M.mlp(256)), (dict(H=264), M.mlp(256)), (dict(), M.mlp(200)),
                      (dict(H=320), M.mlp(256, M.MOE_WEIGHTS_FP8_B128)), (dict(), M.mlp(320, M.MOE_WEIGHTS_W4)),
                      (dict(dtype=M.MOE_DTYPE_FP8_E4M3_B128), M.mlp(256))]:
        p = M.problem(**{**ok, **change})
        scale = None if m.weights == M.MOE_WEIGHTS_BF16 else FAKE
        assert few(M, p, M.gate(), m, us=scale, ds=scale) == M.MOE_ERR_UNSUPPORTED
        assert M.moe_layer_few_workspace_bytes(p, m) == 0


def test_few_buffers(M):
    p, g, bad = M.problem(4, 256, 8, 2, 1, 4), M.gate(), M.MOE_ERR_INVALID_ARG
    bf, w4 = M.mlp(256), M.mlp(256, M.MOE_WEIGHTS_W4, 64)
    assert few(M, None, g, bf) == few(M, p, None, bf) == few(M, p, g, None) == bad
    assert few(M, p, M.gate(groups=3), bf) == bad
    for k in ("x", "logits", "up", "down", "out", "ws"):
        for b in (None, ODD):
            assert few(M, p, g, bf, **{k: b}) == bad, k
    for k in ("bias", "idx", "w"):
        assert few(M, p, g, bf, **{k: ODD}) == bad, k
    assert few(M, p, g, bf, us=FAKE) == few(M, p, g, bf, ds=FAKE) == bad                # scales exactly for scaled weights
    assert few(M, p, g, w4, us=FAKE) == few(M, p, g, w4, ds=FAKE) == few(M, p, g, w4, us=FAKE, ds=ODD) == bad
    assert few(M, p, g, bf, size=M.moe_layer_few_workspace_bytes(p, bf) - 1) == bad
    assert few(M, M.problem(0, 256, 8, 2, 1, 4), g, bf, x=None, logits=None, up=None, down=None, out=None, ws=None,
               size=0) == M.MOE_OK


def test_the_binding_takes_cuda_tensors(M):
    import torch
    t, p = torch.zeros(64, dtype=torch.bfloat16), M.problem(1, 64, 8, 2, 1, 4)
    with pytest.raises(ValueError):
        M.moe_block_norm(p, M.norm(), t, t, t, t, None, t, t)
    with pytest.raises(ValueError):
        M.moe_layer_few(p, M.gate(), M.mlp(64), t, t, None, t, None, t, None, None, None, t, t)
    with pytest.raises(M.MoeError):
        M.run_few_block(M.problem(33, 64, 8, 2, 1, 4), M.gate(), M.mlp(64), M.norm(), *[t] * 11, {}, t, t, t, stream=0)
