"""A block from its normed input to the next block's, as a program runs it: a batch's experts with the join behind the
combine, the same block for a few tokens, and the way back to the router.

Forward: against the composition in 64 bits of the choice that was made. The stages round to bf16 (h; y, where it goes to
memory; r or n), each by at most 2^-8 of the value, and the norms do not magnify: within 4 x 2^-8 of the reference in the
2-norm (fp32 errors are below 2^-14). Backward: every stage against the formulas on the values that it was given."""
import numpy as np
import pytest
import torch

import plain64 as P
import plain64_block as PB

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-6


@pytest.fixture(scope="module")
def M():
    from combine_router_top_gb300 import build as B
    B.build()
    import combine_router_top_gb300 as M
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return M


def rel(a, b):
    return np.linalg.norm(a - b) / np.linalg.norm(b)


def f64(t):
    return t.double().cpu().numpy()


def make(M, T, kind):
    H, inner, E, k, C = 256, 384, 16, 4, 64
    g = torch.Generator(device=DEV).manual_seed(T)
    s = dict(T=T, H=H, E=E, k=k, inner=inner, kind=kind)
    s["p"] = M.problem(T, H, E, k, 4, C)
    s["gate"] = M.gate(M.MOE_SCORE_SIGMOID, 4, 2, M.MOE_GROUP_TOP2, True, 2.5)
    s["x"] = torch.randn((T, H), device=DEV, generator=g).to(torch.bfloat16)
    s["logits"] = torch.randn((T, E), device=DEV, generator=g)
    s["bias"] = 0.1 * torch.randn(E, device=DEV, generator=g)

    def matrix(rows, cols):
        codes = torch.randint(0, 16, (E, rows, cols), dtype=torch.uint8, device=DEV, generator=g)
        scale = ((1 + torch.rand((E, rows, cols // 64), device=DEV, generator=g)) * 0.15 / cols ** 0.5).to(torch.bfloat16)
        return M.w4_pack(codes), scale, f64((codes.double() - 8) * scale.double().repeat_interleave(64, 2))
    s["up"], s["down"] = matrix(2 * inner, H), matrix(H, inner)
    s["residual"] = 2.0 * torch.randn((T, H), device=DEV, generator=g)
    s["w_post"], s["w_pre"] = ((1 + 0.2 * torch.randn(H, device=DEV, generator=g)).to(torch.bfloat16) for _ in range(2))
    s["branch"] = {"none": None, "channel": torch.randn(H, device=DEV, generator=g).to(torch.bfloat16),
                   "token": torch.rand(T, device=DEV, generator=g)}[kind]
    s["norm"] = M.norm(EPS, 0.5, {"none": 0, "channel": 1, "token": 2}[kind], M.MOE_VALUE_F32)
    s["out"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    s["r"], s["n"] = torch.empty_like(s["residual"]), torch.empty_like(s["out"])
    return s


def reference(s, slot=None):
    """r and n from the experts' MLPs of the choice, dropped pairs left out where slot says so."""
    idx, ok, w, _ = P.gate(f64(s["logits"]), f64(s["bias"]), s["k"], 4, 2, True, True, True, 2.5)
    x, y = f64(s["x"]), np.zeros((s["T"], s["H"]))
    for e in range(s["E"]):
        t, j = np.nonzero((idx == e) & ok & (np.ones_like(ok) if slot is None else slot >= 0))
        if len(t):
            y[t] += w[t, j, None] * PB.mlp(x[t], s["up"][2][e], s["down"][2][e], s["inner"])[0]
    r, _, n, _ = PB.forward(y, 0.0, f64(s["residual"]), f64(s["w_post"]), f64(s["w_pre"]),
                            f64(s["branch"]) if s["branch"] is not None else None, s["kind"], 0.5, EPS)
    return idx, ok, y, r, n


@pytest.mark.parametrize("T", [1, 7, 20, 32])
@pytest.mark.parametrize("kind", ["none", "channel", "token"])
def test_few_block(M, T, kind):
    s, bufs = make(M, T, kind), {}
    for _ in range(2):                                  # a second pass finds the workspace as the first left it
        M.run_few_block(s["p"], s["gate"], M.mlp(s["inner"], M.MOE_WEIGHTS_W4, 64), s["norm"], s["x"], s["logits"], s["bias"],
                        s["up"][0], s["up"][1], s["down"][0], s["down"][1], s["residual"], s["w_post"], s["w_pre"],
                        s["branch"], bufs, s["out"], s["r"], s["n"])
    torch.cuda.synchronize()
    assert M.moe_device_status() == M.MOE_OK
    _, _, y, r, n = reference(s)
    assert rel(f64(s["out"]), y) < 2 * 2.0 ** -8
    assert rel(f64(s["r"]), r) < 4 * 2.0 ** -8 and rel(f64(s["n"]), n) < 4 * 2.0 ** -8


@pytest.mark.parametrize("T", [1, 9, 120, 400])
@pytest.mark.parametrize("kind", ["channel", "token"])
def test_w4_block_and_back(M, T, kind):
    s = make(M, T, kind)
    b = M.alloc_buffers(s["p"], DEV)
    h = torch.empty((s["E"], 64, s["inner"]), dtype=torch.bfloat16, device=DEV)
    up = (M.w4(s["H"], s["inner"], 64, M.MOE_ACT_SILU_GATE), *s["up"][:2])
    down = (M.w4(s["inner"], s["H"], 64), *s["down"][:2])
    M.run_w4_block(s["p"], s["gate"], s["norm"], s["x"], s["logits"], s["bias"], up, down, b, h, s["residual"], s["w_post"],
                   s["w_pre"], s["branch"], s["out"], s["r"], s["n"])
    torch.cuda.synchronize()
    assert M.moe_device_status() == M.MOE_OK
    slot = b["slot"].cpu().numpy()
    idx, ok, y, r, n = reference(s, slot)
    assert np.array_equal(b["topk_idx"].cpu().numpy(), idx)
    assert rel(f64(s["out"]), y) < 3 * 2.0 ** -8
    assert rel(f64(s["r"]), r) < 4 * 2.0 ** -8 and rel(f64(s["n"]), n) < 4 * 2.0 ** -8

    g = torch.Generator(device=DEV).manual_seed(T)
    d_r, d_n = torch.randn(s["r"].shape, device=DEV, generator=g), torch.randn(s["n"].shape, device=DEV,
                                                                                generator=g).to(torch.bfloat16)
    f32 = dict(dtype=torch.float32, device=DEV)
    d_out, d_res = torch.empty_like(s["out"]), torch.empty_like(d_r)
    d_post, d_pre = torch.empty(s["H"], **f32), torch.empty(s["H"], **f32)
    d_branch = torch.empty(s["branch"].shape, **f32)
    d_y = torch.zeros((s["E"], 64, s["H"]), dtype=torch.bfloat16, device=DEV)
    d_w, d_l = torch.empty((T, s["k"]), **f32), torch.empty((T, s["E"]), **f32)
    M.run_block_backward(s["p"], s["gate"], s["norm"], s["logits"], s["out"], s["r"], d_r, d_n, s["w_post"], s["w_pre"],
                         s["branch"], b, d_out, d_res, d_post, d_pre, d_branch, d_y, d_w, d_l)
    torch.cuda.synchronize()
    assert M.moe_device_status() == M.MOE_OK
    ref = PB.backward(f64(s["out"]), f64(s["r"]), f64(d_r), f64(d_n), f64(s["w_post"]), f64(s["w_pre"]), f64(s["branch"]),
                      kind, 0.5, EPS)
    for name, got in (("d_y", d_out), ("d_residual", d_res), ("d_w_post", d_post), ("d_w_pre", d_pre), ("d_gate", d_branch)):
        v, bound = ref[name]
        half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
        assert (np.abs(f64(got) - v) <= bound + half * (np.abs(v) + bound)).all(), name
    rows, go = f64(b["y"].view(torch.bfloat16)), f64(d_out)
    w = f64(b["topk_w"])
    dw = np.array([[(go[t] * rows[idx[t, j], slot[t, j]]).sum() if slot[t, j] >= 0 else 0.0 for j in range(s["k"])]
                   for t in range(T)])
    dl, _ = P.gate_backward(f64(s["logits"]), idx, ok, dw, True, True, 2.5)
    assert rel(f64(d_w), dw) < 2.0 ** -14 and rel(f64(d_l), dl) < 2.0 ** -14
    t, j = np.nonzero(slot >= 0)
    assert rel(f64(d_y)[idx[t, j], slot[t, j]], w[t, j, None] * go[t]) < 2.0 ** -8


def test_two_streams_and_a_replayed_block(M):
    """Two blocks at once on two streams with buffers of their own, captured into two graphs and replayed together."""
    sets = [make(M, T, "channel") for T in (5, 12)]
    graphs, streams, want = [], [torch.cuda.Stream() for _ in sets], []

    def go(s, bufs, stream):
        M.run_few_block(s["p"], s["gate"], M.mlp(s["inner"], M.MOE_WEIGHTS_W4, 64), s["norm"], s["x"], s["logits"], s["bias"],
                        s["up"][0], s["up"][1], s["down"][0], s["down"][1], s["residual"], s["w_post"], s["w_pre"],
                        s["branch"], bufs, s["out"], s["r"], s["n"], stream)
    torch.cuda.synchronize()
    for s, stream in zip(sets, streams):
        bufs = {}
        go(s, bufs, stream)
        stream.synchronize()
        want.append([s[n].clone() for n in ("out", "r", "n")])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            go(s, bufs, stream)
        graphs.append(graph)
    for s in sets:
        for n in ("out", "r", "n"):
            s[n].fill_(7)
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for s, w in zip(sets, want):
        assert all(torch.equal(s[n], v) for n, v in zip(("out", "r", "n"), w))
    assert M.moe_device_status() == M.MOE_OK
