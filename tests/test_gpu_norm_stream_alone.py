"""The norm of the residual stream alone (no block before it) and its gradient: every pair of types, rows of one chunk to
the longest, so many rows that a block takes several, any grid."""
import pytest
import torch

import plain64_block as P
from test_gpu_block_norm import DEV, EPS, M, f64, make, near  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H", [(1, 8), (700, 8), (5003, 16), (700, 2056), (640, 7168), (333, 8200), (310, 16384)])
@pytest.mark.parametrize("res,par", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
def test_forward_and_gradient(M, T, H, res, par):
    s = make(M, T, H, "none", res, par, post=False)
    _, _, nn, bn = P.forward(None, 0.0, f64(s["residual"]), None, f64(s["w_pre"]), None, "none", 0.5, EPS)
    refs = {with_dr: P.backward(None, f64(s["residual"]), f64(s["d_r"]) if with_dr else None, f64(s["d_n"]), None,
                                f64(s["w_pre"]), None, "none", 0.5, EPS) for with_dr in (True, False)}
    first = {}
    for blocks in (0, 1, 7):
        p = M.problem(T, H, 1, 1, 1, 1, max_blocks=blocks)
        n = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device=DEV)
        M.moe_block_norm(p, s["norm"], None, s["residual"], None, s["w_pre"], None, None, n)
        got = {"n": n}
        for with_dr in (True, False):
            d_res = torch.full_like(s["residual"], float("nan"))
            d_w = torch.full((H,), float("nan"), device=DEV)
            ws = torch.full((M.moe_block_norm_backward_workspace_bytes(p, s["norm"]),), 0xFF, dtype=torch.uint8, device=DEV)
            M.moe_block_norm_backward(p, s["norm"], None, s["residual"], s["d_r"] if with_dr else None, s["d_n"], None,
                                      s["w_pre"], None, None, d_res, None, d_w, None, ws)
            got["d_residual", with_dr], got["d_w_pre", with_dr] = d_res, d_w
        torch.cuda.synchronize()
        assert M.moe_device_status() == M.MOE_OK
        if not first:
            first = got
            near(n, nn, bn)
            for with_dr, ref in refs.items():
                near(got["d_residual", with_dr], *ref["d_residual"])
                near(got["d_w_pre", with_dr], *ref["d_w_pre"])
        assert all(torch.equal(first[name], got[name]) for name in first)
