"""The norms around a block, alone and behind the combine, and their gradient on the GPU against plain forms in 64 bits.

Tolerance: the bounds derived in plain64_block.py, and one rounding of the result to its type: half a step, 2^-8 of the
value for bf16 and 2^-24 for fp32, and the lowest subnormal's half."""
import numpy as np
import pytest
import torch

import plain64_block as P

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-5
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def M():
    from combine_router_top_gb300 import build as B
    B.build()
    import combine_router_top_gb300 as M
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return M


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def near(got, ref, bound):
    half = HALF[got.dtype]
    err = np.abs(f64(got) - ref)
    bar = bound + half * (np.abs(ref) + bound) + 2.0 ** -133
    assert np.isfinite(f64(got)).all()
    assert (err <= bar).all(), (err / bar).max()


KINDS = {"none": "MOE_BRANCH_PLAIN", "channel": "MOE_BRANCH_CHANNEL", "token": "MOE_BRANCH_TOKEN"}


def make(M, T, H, kind, res, par, post=True, pre=True, scale=0.5, seed=0, extra=()):
    g = torch.Generator(device=DEV).manual_seed(seed + 1000 * T + H)
    rd, pd = (torch.float32 if res == "f32" else torch.bfloat16), (torch.float32 if par == "f32" else torch.bfloat16)

    def rows(dtype, size=1.0):
        return (size * torch.randn((T, H), device=DEV, generator=g)).to(dtype)
    s = {"T": T, "H": H, "kind": kind, "scale": scale}
    s["norm"] = M.norm(EPS, scale, getattr(M, KINDS[kind]), int(res == "f32"), int(par == "f32"))
    s["p"] = M.problem(T, H, 1, 1, 1, 1)
    s["y"], s["residual"] = rows(torch.bfloat16), rows(rd, 3.0)
    s["d_r"], s["d_n"] = rows(rd), rows(torch.bfloat16)
    s["w_post"] = (1 + 0.2 * torch.randn(H, device=DEV, generator=g)).to(pd) if post else None
    s["w_pre"] = (1 + 0.2 * torch.randn(H, device=DEV, generator=g)).to(pd) if pre else None
    s["gate"] = {"none": None, "channel": torch.randn(H, device=DEV, generator=g).to(pd),
                 "token": torch.randn(T, device=DEV, generator=g)}[kind]
    return s


def forward(M, s, stream=None, in_place=False):
    r = s["residual"].clone() if in_place else torch.full_like(s["residual"], float("nan"))
    n = torch.full((s["T"], s["H"]), float("nan"), dtype=torch.bfloat16, device=DEV) if s["w_pre"] is not None else None
    torch.cuda.synchronize()
    M.moe_block_norm(s["p"], s["norm"], s["y"], r if in_place else s["residual"], s["w_post"], s["w_pre"], s["gate"], r,
                     n, stream)
    torch.cuda.synchronize()
    return r, n


def backward(M, s, r, with_dr=True, stream=None, in_place=False, max_blocks=0):
    H, T, f32 = s["H"], s["T"], dict(dtype=torch.float32, device=DEV)
    p = M.problem(T, H, 1, 1, 1, 1, max_blocks=max_blocks)
    o = {"d_y": torch.full_like(s["y"], float("nan"))}
    d_r = s["d_r"].clone() if with_dr else None
    o["d_residual"] = d_r if in_place else torch.full_like(r, float("nan"))
    if s["w_post"] is not None:
        o["d_w_post"] = torch.full((H,), float("nan"), **f32)
    if s["w_pre"] is not None:
        o["d_w_pre"] = torch.full((H,), float("nan"), **f32)
    if s["gate"] is not None:
        o["d_gate"] = torch.full((H if s["kind"] == "channel" else T,), float("nan"), **f32)
    ws = torch.full((M.moe_block_norm_backward_workspace_bytes(p, s["norm"]),), 0xFF, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    M.moe_block_norm_backward(p, s["norm"], s["y"], r, d_r, s["d_n"] if s["w_pre"] is not None else None, s["w_post"],
                              s["w_pre"], s["gate"], o["d_y"], o["d_residual"], o.get("d_w_post"), o.get("d_w_pre"),
                              o.get("d_gate"), ws, stream)
    torch.cuda.synchronize()
    assert M.moe_device_status() == M.MOE_OK
    return o


def check_forward(s, r, n, y=None, dy=0.0):
    rr, br, nn, bn = P.forward(f64(s["y"]) if y is None else y, dy, f64(s["residual"]), f64(s["w_post"]), f64(s["w_pre"]),
                               f64(s["gate"]), s["kind"], s["scale"], EPS)
    near(r, rr, br)
    if n is not None:
        near(n, nn, bn)


def check_backward(s, r, o, with_dr=True):
    ref = P.backward(f64(s["y"]), f64(r), f64(s["d_r"]) if with_dr else None, f64(s["d_n"]), f64(s["w_post"]),
                     f64(s["w_pre"]), f64(s["gate"]), s["kind"], s["scale"], EPS)
    assert set(ref) == set(o)
    for name, (v, b) in ref.items():
        near(o[name], v, b)


SHAPES = [(1, 8), (3, 16), (2, 256), (5, 264), (1, 2048), (7, 2056), (33, 1000), (2, 7168), (3, 8192), (2, 8200),
          (3, 16384)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("res,par", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
def test_forward_and_gradient(M, T, H, kind, res, par):
    s = make(M, T, H, kind, res, par)
    r, n = forward(M, s)
    check_forward(s, r, n)
    check_backward(s, r, backward(M, s, r))


@pytest.mark.parametrize("T,H", [(5, 264), (700, 512), (3, 7168), (2, 12296)])
@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("post,pre", [(False, True), (True, False), (False, False)])
def test_without_one_of_the_norms(M, T, H, kind, post, pre):
    s = make(M, T, H, kind, "bf16", "bf16", post, pre)
    r, n = forward(M, s)
    assert (n is None) == (not pre)
    check_forward(s, r, n)
    check_backward(s, r, backward(M, s, r))


@pytest.mark.parametrize("T,H", [(1, 7168), (19, 264)])
def test_norm_of_the_stream_alone(M, T, H):
    s = make(M, T, H, "none", "f32", "bf16", post=False)
    s["y"] = None
    n = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    M.moe_block_norm(s["p"], s["norm"], None, s["residual"], None, s["w_pre"], None, None, n)
    _, _, nn, bn = P.forward(None, 0.0, f64(s["residual"]), None, f64(s["w_pre"]), None, "none", 0.5, EPS)
    near(n, nn, bn)
    ws = torch.empty(M.moe_block_norm_backward_workspace_bytes(s["p"], s["norm"]), dtype=torch.uint8, device=DEV)
    for d_r in (s["d_r"], None):
        d_res, d_w = torch.empty_like(s["residual"]), torch.empty(H, device=DEV)
        M.moe_block_norm_backward(s["p"], s["norm"], None, s["residual"], d_r, s["d_n"], None, s["w_pre"], None, None, d_res,
                                  None, d_w, None, ws)
        ref = P.backward(None, f64(s["residual"]), f64(d_r), f64(s["d_n"]), None, f64(s["w_pre"]), None, "none", 0.5, EPS)
        near(d_res, *ref["d_residual"])
        near(d_w, *ref["d_w_pre"])


def test_r_alone_or_n_alone(M):
    s = make(M, 6, 520, "channel", "bf16", "bf16")
    r, n = forward(M, s)
    r2, n2 = torch.empty_like(r), torch.empty_like(n)
    M.moe_block_norm(s["p"], s["norm"], s["y"], s["residual"], s["w_post"], None, s["gate"], r2, None)
    M.moe_block_norm(s["p"], s["norm"], s["y"], s["residual"], s["w_post"], s["w_pre"], s["gate"], None, n2)
    assert torch.equal(r, r2) and torch.equal(n, n2)


@pytest.mark.parametrize("T,H,res", [(3001, 256, "f32"), (1021, 2056, "bf16"), (400, 7168, "bf16"), (310, 7168, "f32")])
def test_many_rows(M, T, H, res):
    s = make(M, T, H, "channel", res, "bf16", seed=5)
    r, n = forward(M, s)
    check_forward(s, r, n)
    check_backward(s, r, backward(M, s, r))


@pytest.mark.parametrize("res", ["bf16", "f32"])
def test_in_place_and_capped_grids(M, res):
    """r over the residual, d_residual over d_r; and sums that do not depend on the grid."""
    s = make(M, 977, 1032, "token", res, "bf16")
    r, n = forward(M, s)
    r2, n2 = forward(M, s, in_place=True)
    assert torch.equal(r, r2) and torch.equal(n, n2)
    a = backward(M, s, r)
    for more in (dict(in_place=True), dict(max_blocks=1), dict(max_blocks=7)):
        b = backward(M, s, r, **more)
        assert all(torch.equal(a[k], b[k]) for k in a)


def test_extreme_rows(M):
    """Rows of zeros, of tiny and of huge values, and one of NaN: each row is its own."""
    s = make(M, 6, 2056, "none", "f32", "f32")
    s["y"][0], s["residual"][0] = 0, 0
    s["y"][1] *= 2.0 ** -60
    s["residual"][1] *= 2.0 ** -60
    s["y"][2] *= 2.0 ** 50
    s["residual"][2] *= 2.0 ** 50
    s["y"][3] = float("nan")
    r, n = forward(M, s)
    keep = [0, 1, 2, 4, 5]
    rr, br, nn, bn = P.forward(f64(s["y"])[keep], 0.0, f64(s["residual"])[keep], f64(s["w_post"]), f64(s["w_pre"]), None,
                               "none", 0.5, EPS)
    near(r[keep], rr, br)
    near(n[keep], nn, bn)
    assert r[3].isnan().all() and n[3].isnan().all()
    assert (r[0] == 0).all() and (n[0] == 0).all()


def test_gradient_against_differences(M):
    """Central differences of the forward in 64 bits, along random directions: the formulas themselves."""
    rng = np.random.default_rng(3)
    T, H = 4, 24
    v = {k: rng.standard_normal((T, H)) for k in ("y", "residual", "d_r", "d_n")}
    w = {k: 1 + 0.2 * rng.standard_normal(H) for k in ("w_post", "w_pre")}
    for kind in KINDS:
        gate = rng.standard_normal(T if kind == "token" else H)

        def loss(y, residual, w_post, w_pre, gate):
            r, _, n, _ = P.forward(y, 0.0, residual, w_post, w_pre, gate, kind, 0.5, EPS)
            return (r * v["d_r"]).sum() + (n * v["d_n"]).sum()
        args = {"y": v["y"], "residual": v["residual"], **w, "gate": gate}
        r = P.forward(v["y"], 0.0, v["residual"], w["w_post"], w["w_pre"], gate, kind, 0.5, EPS)[0]
        got = P.backward(v["y"], r, v["d_r"], v["d_n"], w["w_post"], w["w_pre"], gate, kind, 0.5, EPS)
        for name in args:
            if name == "gate" and kind == "none":
                continue
            d = rng.standard_normal(args[name].shape)
            h = 1e-5
            up, down = loss(**{**args, name: args[name] + h * d}), loss(**{**args, name: args[name] - h * d})
            # truncation h^2 times third derivatives of order 10, cancellation 1e-16 * 100 / h
            assert abs((up - down) / (2 * h) - (got["d_" + name][0] * d).sum()) < 1e-7


def routing(M, T, E, k, C, seed, drop_all=()):
    g = torch.Generator(device=DEV).manual_seed(seed)
    top, idx = torch.randn((T, E), device=DEV, generator=g).topk(k, dim=1)
    w = torch.softmax(top, 1)
    i = idx.cpu().numpy()
    slot, used = np.full((T, k), -1, np.int32), np.zeros(E, np.int64)
    for t in range(T):
        for j in range(k):
            if used[i[t, j]] < C and t not in drop_all:
                slot[t, j] = used[i[t, j]]
                used[i[t, j]] += 1
    return idx.to(torch.int32), w, torch.from_numpy(slot).to(DEV), used


@pytest.mark.parametrize("T,H,E,k,C", [(1, 8, 1, 1, 1), (5, 264, 8, 2, 2), (9, 2056, 16, 3, 4), (40, 1032, 64, 6, 3),
                                       (6, 7168, 32, 8, 6), (4, 8192, 16, 5, 4), (3, 12288, 16, 2, 3),
                                       (5, 16384, 64, 16, 5), (7, 520, 20, 12, 7), (300, 256, 4, 4, 300)])
@pytest.mark.parametrize("kind,res,par,post", [("none", "bf16", "bf16", True), ("channel", "f32", "bf16", True),
                                               ("token", "bf16", "f32", False), ("channel", "f32", "f32", True)])
def test_combine_norm(M, T, H, E, k, C, kind, res, par, post):
    s = make(M, T, H, kind, res, par, post)
    lost = {2} if T > 2 else set()                      # a token without a single pair
    idx, w, slot, used = routing(M, T, E, k, C, T + H, lost)
    g = torch.Generator(device=DEV).manual_seed(7)
    y = torch.randn((E, C, H), device=DEV, generator=g).to(torch.bfloat16)
    for e in range(E):
        y[e, int(used[e]):] = float("nan")              # rows of no pair are no inputs
    p = M.problem(T, H, E, k, 1, C)
    out = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device=DEV)
    r, n = torch.full_like(s["residual"], float("nan")), torch.empty_like(out)
    M.moe_combine_norm(p, s["norm"], y, idx, w, slot, s["residual"], s["w_post"], s["w_pre"], s["gate"], out, r, n)
    ref, bound = P.combine(f64(y), idx.cpu().numpy(), f64(w), slot.cpu().numpy())
    near(out, ref, bound)
    check_forward(s, r, n, ref, bound)
    same = torch.empty_like(out)
    M.moe_combine(p, y, idx, w, slot, same)
    assert torch.equal(out, same)
    r2, n2 = s["residual"].clone(), torch.empty_like(n)  # without out, r over the residual
    M.moe_combine_norm(p, s["norm"], y, idx, w, slot, r2, s["w_post"], s["w_pre"], s["gate"], None, r2, n2)
    assert torch.equal(r, r2) and torch.equal(n, n2)


def test_no_rows(M):
    s = make(M, 0, 264, "channel", "bf16", "bf16")
    r, n = torch.empty_like(s["residual"]), torch.empty((0, 264), dtype=torch.bfloat16, device=DEV)
    M.moe_block_norm(s["p"], s["norm"], s["y"], s["residual"], s["w_post"], s["w_pre"], s["gate"], r, n)
    o = backward(M, s, r)
    for name in ("d_w_post", "d_w_pre", "d_gate"):
        assert (o[name] == 0).all()


def test_another_stream_and_a_replayed_graph(M):
    """Forward and gradient on a side stream, captured, replayed on new inputs; rows behind the last stay as they are."""
    s = make(M, 50, 776, "channel", "bf16", "bf16")
    H = 776
    r, n = torch.empty_like(s["residual"]), torch.empty((50, H), dtype=torch.bfloat16, device=DEV)
    d_y = torch.full((52, H), 3.0, dtype=torch.bfloat16, device=DEV)
    d_res, dw, dp, dg = torch.empty_like(r), *(torch.empty(H, device=DEV) for _ in range(3))
    ws = torch.empty(M.moe_block_norm_backward_workspace_bytes(s["p"], s["norm"]), dtype=torch.uint8, device=DEV)

    def go(stream):
        M.moe_block_norm(s["p"], s["norm"], s["y"], s["residual"], s["w_post"], s["w_pre"], s["gate"], r, n, stream)
        M.moe_block_norm_backward(s["p"], s["norm"], s["y"], r, s["d_r"], s["d_n"], s["w_post"], s["w_pre"], s["gate"], d_y,
                                  d_res, dw, dp, dg, ws, stream)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    go(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        go(side)
    for seed in (1, 2):
        new = make(M, 50, H, "channel", "bf16", "bf16", seed=seed)
        for name in ("y", "residual", "d_r", "d_n", "w_post", "w_pre", "gate"):
            s[name].copy_(new[name])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check_forward(s, r, n)
        check_backward(s, r, {"d_y": d_y[:50], "d_residual": d_res, "d_w_post": dw, "d_w_pre": dp, "d_gate": dg})
    assert (d_y[50:] == 3).all() and M.moe_device_status() == M.MOE_OK
