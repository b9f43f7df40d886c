"""The norms around a block with many rows to a thread block: rings that turn many times, tokens without pairs, every row
length's kernel, and grids of one block. Bounds as for few rows."""
import pytest
import torch

import plain64_block as P
from test_gpu_block_norm import DEV, M, backward, check_backward, check_forward, f64, forward, make, near, routing  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,E,k,C", [(304, 2056, 16, 3, 40), (333, 2064, 8, 8, 400), (700, 4096, 64, 2, 30), (310, 7168, 32, 8, 90),
                                       (305, 8200, 16, 5, 100), (320, 16384, 64, 16, 100), (304, 2304, 4, 1, 20)])
@pytest.mark.parametrize("kind,res,par,post", [("none", "bf16", "bf16", True), ("channel", "f32", "bf16", True),
                                               ("token", "bf16", "f32", False)])
def test_combine_norm_of_many_tokens(M, T, H, E, k, C, kind, res, par, post):
    s = make(M, T, H, kind, res, par, post)
    idx, w, slot, used = routing(M, T, E, k, C, T + H, {0, 2, 3, T - 1} | set(range(150, 170)))
    g = torch.Generator(device=DEV).manual_seed(7)
    y = torch.randn((E, C, H), device=DEV, generator=g).to(torch.bfloat16)
    for e in range(E):
        y[e, int(used[e]):] = float("nan")              # rows of no pair are no inputs
    ref, bound = P.combine(f64(y), idx.cpu().numpy(), f64(w), slot.cpu().numpy())
    first = None
    for blocks in (0, 1, 7):
        p = M.problem(T, H, E, k, 1, C, max_blocks=blocks)
        out = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device=DEV)
        r, n = torch.full_like(s["residual"], float("nan")), torch.empty_like(out)
        M.moe_combine_norm(p, s["norm"], y, idx, w, slot, s["residual"], s["w_post"], s["w_pre"], s["gate"], out, r, n)
        torch.cuda.synchronize()
        assert M.moe_device_status() == M.MOE_OK
        if first is None:
            first = out, r, n
            near(out, ref, bound)
            check_forward(s, r, n, ref, bound)
            same = torch.empty_like(out)
            M.moe_combine(p, y, idx, w, slot, same)
            assert torch.equal(out, same)
        assert all(torch.equal(a, b) for a, b in zip(first, (out, r, n)))
    r2, n2 = s["residual"].clone(), torch.empty_like(first[2])         # without out, r over the residual
    M.moe_combine_norm(p, s["norm"], y, idx, w, slot, r2, s["w_post"], s["w_pre"], s["gate"], None, r2, n2)
    assert torch.equal(first[1], r2) and torch.equal(first[2], n2)


@pytest.mark.parametrize("T,H", [(608, 8), (640, 256), (609, 2056), (611, 5128), (608, 7176), (610, 8192), (608, 8200), (300, 4104)])
@pytest.mark.parametrize("kind,res,par,post", [("none", "f32", "bf16", True), ("channel", "bf16", "f32", True),
                                               ("token", "f32", "f32", False), ("channel", "bf16", "bf16", True)])
def test_many_rows_on_any_grid(M, T, H, kind, res, par, post):
    s = make(M, T, H, kind, res, par, post)
    r, n = forward(M, s)
    check_forward(s, r, n)
    a = backward(M, s, r)
    check_backward(s, r, a)
    for blocks in (1, 9):
        r2, n2 = forward(M, {**s, "p": M.problem(T, H, 1, 1, 1, 1, max_blocks=blocks)})
        assert torch.equal(r, r2) and torch.equal(n, n2)
        b = backward(M, s, r, max_blocks=blocks)
        assert all(torch.equal(a[name], b[name]) for name in a)
    assert M.moe_device_status() == M.MOE_OK


def test_two_calls_at_once(M):
    """The same inputs by two streams at once, each with outputs and a workspace of its own."""
    s = make(M, 700, 4104, "channel", "bf16", "bf16")
    r, n = forward(M, s)
    want = backward(M, s, r)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    size = M.moe_block_norm_backward_workspace_bytes(s["p"], s["norm"])
    made = []
    for stream in streams:
        with torch.cuda.stream(stream):
            f32 = dict(dtype=torch.float32, device=DEV)
            o = dict(r=torch.empty_like(r), n=torch.empty_like(n), d_y=torch.empty_like(n), d_residual=torch.empty_like(r),
                     **{name: torch.empty(4104, **f32) for name in ("d_w_post", "d_w_pre", "d_gate")},
                     ws=torch.empty(size, dtype=torch.uint8, device=DEV))
        made.append(o)
    torch.cuda.synchronize()
    for _ in range(3):
        for stream, o in zip(streams, made):
            M.moe_block_norm(s["p"], s["norm"], s["y"], s["residual"], s["w_post"], s["w_pre"], s["gate"], o["r"], o["n"], stream)
            M.moe_block_norm_backward(s["p"], s["norm"], s["y"], o["r"], s["d_r"], s["d_n"], s["w_post"], s["w_pre"], s["gate"],
                                      o["d_y"], o["d_residual"], o["d_w_post"], o["d_w_pre"], o["d_gate"], o["ws"], stream)
    torch.cuda.synchronize()
    for o in made:
        assert torch.equal(o["r"], r) and torch.equal(o["n"], n)
        assert all(torch.equal(o[name], want[name]) for name in ("d_y", "d_residual", "d_w_post", "d_w_pre", "d_gate"))


@pytest.mark.parametrize("T,H", [(5, 264), (9, 4104), (6, 7168), (3, 12296)])
@pytest.mark.parametrize("kind", ["none", "channel", "token"])
def test_a_gradient_along_the_row(M, T, H, kind):
    """w_pre d_n along r, up to its rounding: the norm's gradient cancels, and with it the mean over D, which the kernel takes
    from sums of D's parts."""
    s = make(M, T, H, kind, "f32", "bf16")
    r, _ = forward(M, s)
    s["d_n"] = (r / s["w_pre"].float()).to(torch.bfloat16)
    check_backward(s, r, backward(M, s, r, with_dr=False), with_dr=False)
    s["d_r"] *= 2.0 ** -12
    check_backward(s, r, backward(M, s, r))
