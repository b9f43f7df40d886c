"""The gated route, the 4-bit experts, the combine and the way back, run together as a program runs them.

Forward: against the composition in 64 bits of the choice that was made. The stages round to bf16 at h, y and out, each
by at most 2^-9 of the value, so that the output is within 3 x 2^-8 of the reference in the 2-norm (the silu's and the
down product's slopes are near 1 on this data; the sums' own fp32 errors are below 2^-16). With fp8 rows the reference
takes the dequantised codes.
Backward: d_topk_w and d_logits are fp32 throughout: 2^-14 in the 2-norm."""
import numpy as np
import pytest
import torch

import plain64 as P

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def M():
    from combine_router_top_gb300 import build as B
    B.build()
    import combine_router_top_gb300 as M
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return M


def rel(a, b):
    return np.linalg.norm(a - b) / np.linalg.norm(b)


@pytest.mark.parametrize("T", [1, 9, 120])
@pytest.mark.parametrize("fp8", [False, True])
def test_forward_and_back(M, T, fp8):
    H, inner, E, k, C = 256, 384, 16, 4, 64
    g = torch.Generator(device=DEV).manual_seed(T + fp8)
    p = M.problem(T, H, E, k, 4, C, int(fp8))
    gate = M.gate(M.MOE_SCORE_SIGMOID, 4, 2, M.MOE_GROUP_TOP2, True, 2.5)
    x = torch.randn((T, H), device=DEV, generator=g).to(torch.bfloat16)
    logits = torch.randn((T, E), device=DEV, generator=g)
    bias = 0.1 * torch.randn(E, device=DEV, generator=g)

    def matrix(rows, cols, group):
        codes = torch.randint(0, 16, (E, rows, cols), dtype=torch.uint8, device=DEV, generator=g)
        scale = ((1 + torch.rand((E, rows, cols // group), device=DEV, generator=g)) * 0.15 / cols ** 0.5).to(torch.bfloat16)
        return codes, scale
    cu, su = matrix(2 * inner, H, 64)
    cd, sd = matrix(H, inner, 128)
    up = (M.w4(H, inner, 64, M.MOE_ACT_SILU_GATE), M.w4_pack(cu), su)
    down = (M.w4(inner, H, 128), M.w4_pack(cd), sd)
    b = M.alloc_buffers(p, DEV)
    h = torch.empty((E, C, inner), dtype=torch.bfloat16, device=DEV)
    out = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    for _ in range(2):                                  # a second pass finds the buffers as the first left them
        M.run_w4_path(p, gate, x, logits, bias, up, down, b, h, out)
    torch.cuda.synchronize()
    assert M.moe_device_status() == M.MOE_OK
    idx, ok, w, _ = P.gate(logits.cpu().numpy(), bias.double().cpu().numpy(), k, 4, 2, True, True, True, 2.5)
    assert np.array_equal(b["topk_idx"].cpu().numpy(), idx) and ok.all()
    xs = x.double().cpu().numpy()
    if fp8:
        rows = b["recv"].view(torch.float8_e4m3fn).double() * b["recv_scale"].double().repeat_interleave(128, 2)
    ref = np.zeros((T, H))
    y = b["y"].view(torch.bfloat16).double().cpu().numpy()
    for t in range(T):
        for j in range(k):
            e, s = idx[t, j], int(b["slot"][t, j])
            if s < 0:                                   # past its expert's capacity: the combine leaves it out
                continue
            v = rows[e, s].cpu().numpy() if fp8 else xs[t]
            r, _ = P.w4_rows(v[None], cu[e].cpu().numpy(), su[e].double().cpu().numpy(), 64)
            a = P.silu(r[:, :inner]) * r[:, inner:]
            r, _ = P.w4_rows(a, cd[e].cpu().numpy(), sd[e].double().cpu().numpy(), 128)
            ref[t] += w[t, j] * r[0]
    assert rel(out.double().cpu().numpy(), ref) < 3 * 2.0 ** -8

    d_out = torch.randn((T, H), device=DEV, generator=g).to(torch.bfloat16)
    d_y = torch.zeros((E, C, H), dtype=torch.bfloat16, device=DEV)
    d_w, d_l = torch.empty((T, k), device=DEV), torch.empty((T, E), device=DEV)
    M.run_gate_backward(p, gate, logits, d_out, b, d_y, d_w, d_l)
    torch.cuda.synchronize()
    slot = b["slot"].cpu().numpy()
    go = d_out.double().cpu().numpy()
    dw = np.array([[(go[t] * y[idx[t, j], slot[t, j]]).sum() if slot[t, j] >= 0 else 0.0 for j in range(k)]
                   for t in range(T)])
    dl, _ = P.gate_backward(logits.cpu().numpy(), idx, ok, dw, True, True, 2.5)
    assert rel(d_w.double().cpu().numpy(), dw) < 2.0 ** -14
    assert rel(d_l.double().cpu().numpy(), dl) < 2.0 ** -14


def test_buffers_of_a_larger_batch_serve_smaller_ones_and_larger_again(M):
    """The path's workspace grows with the problem that needs more of it."""
    H, E, k, C = 128, 4, 2, 32
    g = torch.Generator(device=DEV).manual_seed(7)
    w = (M.w4(H, H, 64), torch.randint(0, 256, (E, H, H // 2), dtype=torch.uint8, device=DEV, generator=g),
         torch.full((E, H, H // 64), 0.02, dtype=torch.bfloat16, device=DEV))
    x = torch.randn((40, H), device=DEV, generator=g).to(torch.bfloat16)
    logits = torch.randn((40, E), device=DEV, generator=g)
    b = M.alloc_buffers(M.problem(40, H, E, k, 1, C, 1), DEV)
    h = torch.empty((E, C, H), dtype=torch.bfloat16, device=DEV)
    outs = {}
    for T in (2, 40, 2, 40):
        out = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
        M.run_w4_path(M.problem(T, H, E, k, 1, C, 1), M.gate(), x, logits, None, w, w, b, h, out)
        torch.cuda.synchronize()
        assert torch.equal(outs.setdefault(T, out), out)
    assert rel(outs[40][:2].double().cpu().numpy(), outs[2].double().cpu().numpy()) < 3 * 2.0 ** -8
