"""The whole layer for a few tokens on the GPU against a plain form in 64 bits: the choice as plain64.gate makes it, the
experts' MLPs with h rounded as the layer's definition has it.

Tolerance: plain64_block.mlp's bound for each pair, weighted; the weighted sum's own roundings, 2 for each of at most 17
terms and 3 for the warps' joining, 2^-19 of the sum of magnitudes with room; a routing weight's own error, 2^-20 of it
(test_gpu_gate.py's); and one rounding to bf16, 2^-8 of the value."""
import numpy as np
import pytest
import torch

import plain64 as P
import plain64_block as PB

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def M():
    from combine_router_top_gb300 import build as B
    B.build()
    import combine_router_top_gb300 as M
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return M


def matrix(M, n, rows, cols, kind, group, g):
    """(weights, scales, their values [n][rows][cols] in float64, for 4-bit ones their operands' magnitudes)"""
    if kind == "bf16":
        w = (torch.randn((n, rows, cols), device=DEV, generator=g) / cols ** 0.5).to(torch.bfloat16)
        return w, None, w.double().cpu().numpy(), None
    if kind == "fp8":
        q = torch.randint(0, 256, (n, rows, cols), dtype=torch.uint8, device=DEV, generator=g)
        q = torch.where((q & 0x7F) == 0x7F, q - 1, q)        # every code but the NaNs
        s = (1 + torch.rand((n, rows // 128, cols // 128), device=DEV, generator=g)) * 0.01 / cols ** 0.5
        v = q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 1).repeat_interleave(128, 2)
        return q, s, v.cpu().numpy(), None
    q = torch.randint(0, 16, (n, rows, cols), dtype=torch.uint8, device=DEV, generator=g)
    s = ((1 + torch.rand((n, rows, cols // group), device=DEV, generator=g)) * 0.15 / cols ** 0.5).to(torch.bfloat16)
    full = s.double().repeat_interleave(group, 2)
    return M.w4_pack(q), s, ((q.double() - 8) * full).cpu().numpy(), (1040 * full).cpu().numpy()


def make(M, T, E, k, H, I, kind, group=128, shared=0, seed=0, sigmoid=True, logits_bf16=False):
    g = torch.Generator(device=DEV).manual_seed(seed + 7 * T + H)
    s = dict(T=T, E=E, k=k, H=H, I=I, shared=shared, sigmoid=sigmoid, kind=kind)
    s["x"] = torch.randn((T, H), device=DEV, generator=g).to(torch.bfloat16)
    s["logits"] = torch.randn((T, E), device=DEV, generator=g)
    if logits_bf16:
        s["logits"] = s["logits"].to(torch.bfloat16)
    s["bias"] = 0.1 * torch.randn(E, device=DEV, generator=g) if sigmoid else None
    s["gate"] = M.gate(M.MOE_SCORE_SIGMOID if sigmoid else M.MOE_SCORE_SOFTMAX, scale=1.5,
                       logits_type=M.MOE_LOGITS_BF16 if logits_bf16 else M.MOE_LOGITS_F32)
    s["mlp"] = M.mlp(I, {"bf16": M.MOE_WEIGHTS_BF16, "fp8": M.MOE_WEIGHTS_FP8_B128, "w4": M.MOE_WEIGHTS_W4}[kind], group, shared)
    s["up"] = matrix(M, E + shared, 2 * I, H, kind, group, g)
    s["down"] = matrix(M, E + shared, H, I, kind, group, g)
    return s


def run(M, s, stream=None, max_blocks=0, lists=True, out=None):
    T, H, k = s["T"], s["H"], s["k"]
    p = M.problem(T, H, s["E"], k, 1, 1, max_blocks=max_blocks)
    idx = torch.full((T, k), -7, dtype=torch.int32, device=DEV) if lists else None
    w = torch.full((T, k), float("nan"), device=DEV) if lists else None
    out = torch.full((T + 1, H), 3.0, dtype=torch.bfloat16, device=DEV) if out is None else out
    ws = torch.full((M.moe_layer_few_workspace_bytes(p, s["mlp"]),), 0xFF, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    M.moe_layer_few(p, s["gate"], s["mlp"], s["x"], s["logits"], s["bias"], s["up"][0], s["up"][1], s["down"][0],
                    s["down"][1], idx, w, out[:T], ws, stream)
    torch.cuda.synchronize()
    assert M.moe_device_status() == M.MOE_OK
    assert (out[T:] == 3).all()
    return idx, w, out[:T]


def check(s, idx, w, out):
    T, E, k, I = s["T"], s["E"], s["k"], s["I"]
    bias = s["bias"].double().cpu().numpy() if s["bias"] is not None else None
    ri, ok, rw, _ = P.gate(s["logits"].double().cpu().numpy(), bias, k, sigmoid=s["sigmoid"], scale=1.5)
    if idx is not None:
        assert (idx.cpu().numpy()[ok] == ri[ok]).all()
        assert np.abs(w.double().cpu().numpy() - rw).max() <= 2.0 ** -20 * 1.5
        assert (w.cpu().numpy()[~ok] == 0).all()
    x = s["x"].double().cpu().numpy()
    ref, bound, mag = np.zeros((T, s["H"])), np.zeros((T, s["H"])), np.zeros((T, s["H"]))
    for e in range(E + s["shared"]):
        t, j = np.nonzero((ri == e) & ok) if e < E else (np.arange(T), None)
        if len(t) == 0:
            continue
        v, B = PB.mlp(x[t], s["up"][2][e], s["down"][2][e], I, s["kind"] != "bf16",
                      *(m[3][e] if m[3] is not None else None for m in (s["up"], s["down"])))
        by = rw[t, j][:, None] if j is not None else 1.0
        ref[t] += by * v
        bound[t] += np.abs(by) * B
        mag[t] += np.abs(by * v)
    o = out.double().cpu().numpy()
    bar = bound + (2.0 ** -19 + 2.0 ** -20) * mag + 2.0 ** -8 * np.abs(ref) + 2.0 ** -133
    err = np.abs(o - ref)
    assert np.isfinite(o).all()
    assert (err <= bar).all(), (err / bar).max()
    # the bounds add worst cases up; what is left in earnest is the output's rounding, at most 2^-8 of each value
    assert np.linalg.norm(err) <= (2.0 ** -8 + 2.0 ** -12) * np.linalg.norm(ref)


def steps(kind):
    return 64 if kind == "bf16" else 128


KINDS = [("bf16", 128), ("fp8", 128), ("w4", 32), ("w4", 64), ("w4", 128)]


@pytest.mark.parametrize("kind,group", KINDS)
@pytest.mark.parametrize("T,E,k", [(1, 4, 2), (2, 1, 1), (3, 8, 2), (8, 8, 3), (9, 3, 2), (16, 4, 4), (17, 2, 1), (25, 16, 4),
                                   (32, 1, 1), (32, 64, 8), (31, 24, 16)])
def test_small_layers(M, T, E, k, kind, group):
    """One row to 32 for an expert, with and without the shared one."""
    u = steps(kind)
    for shared in (0, 1):
        s = make(M, T, E, k, 3 * u, 2 * u, kind, group, shared, sigmoid=E % 3 != 0)
        check(s, *run(M, s))


@pytest.mark.parametrize("kind,group", KINDS)
@pytest.mark.parametrize("T,H,I", [(1, 1, 1), (5, 2176, 128), (3, 384, 2176), (12, 4224, 640), (2, 1152, 4736)])
def test_long_and_ragged_inputs(M, T, H, I, kind, group):
    """Rows of one piece and of several, whose last one is short for some warps and empty for others."""
    u = steps(kind)
    s = make(M, T, 4, 2, max(H, u), max(I, u), kind, group, 1)
    check(s, *run(M, s))


def test_odd_multiples_of_64(M):
    for T, H, I in ((4, 64, 320), (11, 832, 64), (3, 1088, 576)):
        s = make(M, T, 6, 2, H, I, "bf16", shared=1)
        check(s, *run(M, s))


@pytest.mark.parametrize("E,G,top,rule,logits_bf16", [(256, 8, 4, 1, False), (160, 8, 3, 0, True), (1024, 1, 1, 0, False),
                                                      (1000, 20, 7, 1, False), (100, 1, 1, 0, True)])
def test_gates(M, E, G, top, rule, logits_bf16):
    """The choice is the gated route's, whatever its lanes hold."""
    s = make(M, 6, E, 6, 128, 64, "bf16", logits_bf16=logits_bf16)
    s["gate"] = M.gate(M.MOE_SCORE_SIGMOID, G, top, rule, True, 1.5, int(logits_bf16))
    idx, w, out = run(M, s)
    p = M.problem(6, 128, E, 6, 1, 16)
    b = M.alloc_buffers(p, DEV)
    M.moe_route_gated(p, s["gate"], s["logits"], s["bias"], b["topk_idx"], b["topk_w"], b["counts"], b["offsets"], b["slot"],
                      b["rank_counts"], b["dropped"], b["workspace"])
    torch.cuda.synchronize()
    assert torch.equal(idx, b["topk_idx"]) and torch.equal(w, b["topk_w"])
    x, ri, rw = s["x"].double().cpu().numpy(), idx.cpu().numpy(), w.double().cpu().numpy()
    for t in range(6):
        v = sum(rw[t, j] * PB.mlp(x[t:t + 1], s["up"][2][ri[t, j]], s["down"][2][ri[t, j]], 64)[0][0] for j in range(6))
        assert np.linalg.norm(out[t].double().cpu().numpy() - v) < 2.0 ** -7 * np.linalg.norm(v)


@pytest.mark.parametrize("shared", [0, 1])
def test_masked_logits(M, shared):
    """Tokens with fewer experts than choices, one with none, one whose only expert is alone with it."""
    s = make(M, 5, 8, 3, 128, 64, "bf16", shared=shared)
    s["logits"][1, 2:] = -float("inf")
    s["logits"][2, :] = float("nan")
    s["logits"][3, :] = -3.4e38
    s["logits"][3, 7] = 0.5
    s["logits"][4, 7] = -float("inf")
    idx, w, out = run(M, s)
    check(s, idx, w, out)
    if not shared:
        assert (out[2] == 0).all()
    s["logits"][:] = -float("inf")                       # not one pair in the batch
    idx, w, out = run(M, s)
    check(s, idx, w, out)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "w4"])
def test_other_experts_and_tokens_do_not_matter(M, kind):
    """Weights that no token chose may hold anything, and a token's row of infinities stays its own."""
    u = steps(kind)
    s = make(M, 4, 16, 2, 2 * u, u, kind, 64)
    idx, _, out = run(M, s)
    for e in set(range(16)) - set(idx.flatten().tolist()):
        for m in ("up", "down"):
            if kind == "bf16":
                s[m][0][e] = float("nan")
            else:
                s[m][1][e] = float("nan")
    assert torch.equal(run(M, s)[2], out)
    s["x"][1] = float("inf")
    again = run(M, s)[2]
    assert torch.equal(again[[0, 2, 3]], out[[0, 2, 3]]) and not torch.isfinite(again[1].float()).any()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "w4"])
def test_repeatable_on_any_grid(M, kind):
    s = make(M, 13, 16, 4, 512, 384, kind, 32, 1)
    idx, w, out = run(M, s)
    for more in (dict(), dict(max_blocks=1), dict(max_blocks=5), dict(lists=False), dict(stream=torch.cuda.Stream())):
        again = run(M, s, **more)
        assert torch.equal(again[2], out)


def test_no_tokens(M):
    s = make(M, 0, 8, 2, 128, 64, "bf16")
    run(M, s)


@pytest.mark.parametrize("kind", ["bf16", "w4"])
def test_layers_in_a_row_and_replayed(M, kind):
    """Two layers behind one another, the second on the first's output, on one workspace, captured and replayed on new
    inputs: what a decode step does."""
    u = steps(kind)
    s1, s2 = (make(M, 3, 8, 2, 4 * u, 2 * u, kind, 64, 1, seed=i) for i in (1, 2))
    p = M.problem(3, 4 * u, 8, 2, 1, 1)
    ws = torch.empty(M.moe_layer_few_workspace_bytes(p, s1["mlp"]), dtype=torch.uint8, device=DEV)
    mid, out = (torch.empty((3, 4 * u), dtype=torch.bfloat16, device=DEV) for _ in range(2))

    def go(stream):
        for s, i, o in ((s1, s1["x"], mid), (s2, mid, out)):
            M.moe_layer_few(p, s["gate"], s["mlp"], i, s["logits"], s["bias"], s["up"][0], s["up"][1], s["down"][0],
                            s["down"][1], None, None, o, ws, stream)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    go(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        go(side)
    for seed in (5, 6):
        new = make(M, 3, 8, 2, 4 * u, 2 * u, kind, 64, 1, seed=seed)
        s1["x"].copy_(new["x"])
        s1["logits"].copy_(new["logits"])
        torch.cuda.synchronize()
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        check(s1, None, None, mid)
        check({**s2, "x": mid}, None, None, out)
    assert M.moe_device_status() == M.MOE_OK
