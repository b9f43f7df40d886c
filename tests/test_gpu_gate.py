"""The gated route and its gradient on the GPU against a plain form in 64 bits.

Choice. Keys are fp32: sigmoid takes four roundings (exp within 2 ulp, sum, division) and the bias one more, so that a
key is within 8 ulp of 2 + |b| or 2^-21 (2 + |b|) of its 64-bit value, group sums of two within twice that. A token
whose 64-bit margin is under 2^-18 (for |b| <= 1) may choose otherwise; such tokens are left out (and must be few).
Unbiased keys are the logits themselves: every token has to agree.
Weights: score within 8 roundings (softmax sums of up to 1024 terms compensated), quotient and scale 2, a sum over k
<= 16 terms 4 + exp 2: 16 x 2^-24 relative, 2^-20.
Gradient: with the magnitude that an element is formed from (plain64.gate_backward), 16 roundings for w, s and the dot
product, and for a softmax over E experts E/32 + 16 more in its sum: (48 + E/32) 2^-24 of it; bf16 adds 2^-8 of the
value (half an ulp is 2^-9)."""
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


def gate_of(M, c, bf16):
    return M.gate(M.MOE_SCORE_SIGMOID if c["sigmoid"] else M.MOE_SCORE_SOFTMAX, c["G"], c["top_g"],
                  M.MOE_GROUP_TOP2 if c["top2"] else M.MOE_GROUP_MAX, c["renorm"], c["scale"],
                  M.MOE_LOGITS_BF16 if bf16 else M.MOE_LOGITS_F32)


def on_device(l, bf16):
    t = torch.from_numpy(np.ascontiguousarray(l, dtype=np.float32)).to(DEV)
    return t.to(torch.bfloat16) if bf16 else t


def route(M, l, bias, k, c, R=1, C=1 << 20, bf16=False, stream=None):
    T, E = l.shape
    p = M.problem(T, 8, E, k, R, C)
    i32 = dict(dtype=torch.int32, device=DEV)
    o = {"topk_idx": torch.full((T, k), -7, **i32), "topk_w": torch.full((T, k), -7.0, device=DEV),
         "counts": torch.full((E,), -7, **i32), "offsets": torch.full((E + 1,), -7, **i32),
         "slot": torch.full((T, k), -7, **i32), "rank_counts": torch.full((R,), -7, **i32),
         "dropped": torch.full((1,), -7, **i32)}
    ws = torch.full((M.moe_route_workspace_bytes(p),), 0x55, dtype=torch.uint8, device=DEV)
    b = None if bias is None else torch.from_numpy(np.asarray(bias, np.float32)).to(DEV)
    x = on_device(l, bf16)
    torch.cuda.synchronize()                            # the inputs are made on the default stream
    M.moe_route_gated(p, gate_of(M, c, bf16), x, b, *o.values(), ws, stream=stream)
    torch.cuda.synchronize()
    return {n: v.cpu().numpy() for n, v in o.items()}


def check(M, l, bias, k, c, R=1, C=1 << 20, bf16=False, exact=False):
    """The route against the plain form. exact: keys have no rounding, so every choice has to agree."""
    l = P.bf16_round(l) if bf16 else np.asarray(l, np.float32)
    got = route(M, l, bias, k, c, R, C, bf16)
    b64 = None if bias is None else np.asarray(bias, np.float32).astype(np.float64)
    idx, ok, w, margin = P.gate(l, b64, k, **c)
    # an unbiased choice among groups ranked by sums of scores rounds in those sums only
    sure = np.full(len(l), True) if exact else margin > 2.0 ** -18
    assert sure.mean() > 0.9
    assert np.array_equal(got["topk_idx"][sure], idx[sure])
    assert np.allclose(got["topk_w"][sure], w[sure], rtol=2.0 ** -20, atol=1e-37)
    if not sure.all():                                   # whatever was chosen, it is counted as chosen
        idx = got["topk_idx"]
    ref = P.count(idx, ok, l.shape[1], R, C)
    for n in ("counts", "offsets", "slot", "rank_counts"):
        assert np.array_equal(got[n], ref[n]), n
    assert got["dropped"][0] == ref["dropped"]
    for row in got["topk_idx"]:
        assert len(set(row)) == k and 0 <= row.min() and row.max() < l.shape[1]
    return got, ok


BASE = dict(G=1, top_g=1, top2=False, sigmoid=True, renorm=True, scale=1.0)
SHAPES = {
    # (T, E, k, R, C, gate): one token, one tile, one more, tiles of 8, tiles of 32, ragged ends
    "one": (1, 256, 8, 8, 16, dict(G=8, top_g=4, top2=True, scale=2.5)),
    "T31": (31, 64, 6, 4, 5, dict(renorm=False)),
    "T32": (32, 64, 6, 4, 5, dict(sigmoid=False)),
    "T33": (33, 64, 6, 4, 5, dict(sigmoid=False, renorm=False, scale=16.0)),
    "T1025": (1025, 256, 8, 8, 30, dict(G=8, top_g=4, top2=True, scale=2.5)),
    "T1300_two_level": (4100, 256, 2, 8, 64, dict(G=4, top_g=2)),
    # experts that no lane count divides, groups that the warp does not divide into, one expert, many
    "E1": (9, 1, 1, 1, 4, dict(renorm=False)),
    "E6_G3": (50, 6, 3, 3, 50, dict(G=3, top_g=2)),
    "E35_G5": (77, 35, 7, 5, 40, dict(G=5, top_g=1, top2=True)),
    "E160_G8": (100, 160, 6, 8, 40, dict(G=8, top_g=3, sigmoid=False, renorm=False, scale=16.0)),
    "E372_G31": (40, 372, 16, 31, 9, dict(G=31, top_g=9, top2=True)),
    "E1003_G17": (34, 1003, 16, 17, 3, dict(G=17, top_g=5, top2=True, sigmoid=False)),
    "E1024": (70, 1024, 16, 8, 3, dict()),
    "E1024_G32": (40, 1024, 1, 32, 3, dict(G=32, top_g=32, top2=True, renorm=False)),
    "k_is_all_of_the_groups": (20, 24, 6, 4, 30, dict(G=8, top_g=2, sigmoid=False)),
    "negative_scale": (12, 16, 4, 2, 30, dict(scale=-0.5)),
}


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("name", SHAPES)
def test_route(M, name, biased, bf16):
    T, E, k, R, C, more = SHAPES[name]
    c = {**BASE, **more}
    rng = np.random.default_rng(sum(map(ord, name)) + 2 * biased + bf16)
    l = rng.standard_normal((T, E))
    bias = 0.3 * rng.standard_normal(E) if biased else None
    check(M, l, bias, k, c, R, C, bf16, exact=not biased and not (c["G"] > 1 and c["top2"]))


@pytest.mark.parametrize("T", [5, 40, 2000])
def test_ties_go_to_the_lowest_index(M, T):
    """sigmoid(0) + b is exact for b a multiple of 1/8, and so are sums of two: all keys and group scores tie often."""
    rng = np.random.default_rng(T)
    E = 48
    bias = rng.integers(-3, 4, E) / 8.0
    check(M, np.zeros((T, E)), bias, 5, {**BASE, "G": 6, "top_g": 3, "top2": True}, 1, 1 << 20, exact=True)
    l = rng.integers(0, 3, (T, E)).astype(np.float64)
    l[l == 0] = np.where(rng.random((l == 0).sum()) < 0.5, 0.0, -0.0)
    check(M, l, None, 5, {**BASE, "G": 6, "top_g": 3, "sigmoid": False}, 1, 1 << 20, exact=True)


LOW_F32, LOW_BF16 = -3.4028234663852886e38, P.MASK_LOGIT


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("mask", [-np.inf, np.nan, LOW_F32, LOW_BF16])
def test_masked_experts_are_no_pairs(M, mask, renorm, sigmoid):
    """Rows with fewer open experts than k, with none at all, and groups that the mask leaves empty."""
    rng = np.random.default_rng(3)
    T, E, k = 70, 32, 6
    l = rng.standard_normal((T, E))
    l[rng.random((T, E)) < 0.85] = mask
    l[7] = mask
    l[8, 1:] = mask
    for bias in (None, 0.25 * rng.standard_normal(E)):
        for c in (dict(), dict(G=4, top_g=2), dict(G=4, top_g=2, top2=True)):
            c = {**BASE, "sigmoid": sigmoid, "renorm": renorm, **c}
            got, ok = check(M, l, bias, k, c, 2, 20, exact=False)
            assert (got["slot"][~ok] == -1).all() and (got["topk_w"][~ok] == 0).all()
            assert not ok[7].any() and ok[8].sum() <= 1
            if mask == LOW_BF16:
                check(M, l, bias, k, c, 2, 20, bf16=True)


def test_bias_of_minus_infinity_takes_an_expert_out(M):
    rng = np.random.default_rng(4)
    l = rng.standard_normal((300, 64))
    bias = 0.1 * rng.standard_normal(64)
    bias[[3, 17, 40]] = -np.inf
    bias[41] = np.nan
    for s in (True, False):
        got, ok = check(M, l, bias, 8, {**BASE, "sigmoid": s}, 4, 64)
        assert ok.all() and got["counts"][[3, 17, 40, 41]].sum() == 0


def test_infinite_and_extreme_logits(M):
    l = np.zeros((40, 16))
    l[:, 3], l[:, 5] = np.inf, np.inf
    l[1] = -200.0                                       # every sigmoid underflows: weights of 0
    l[2] = 200.0
    l[3, :] = -1e30
    for c in (dict(), dict(sigmoid=False), dict(sigmoid=False, renorm=False), dict(renorm=False)):
        c = {**BASE, **c}
        got, _ = check(M, l, None, 4, c, 1, 64, exact=True)
        assert np.isfinite(got["topk_w"]).all()
    l[1:] = 0.0
    l[0] = np.arange(16) * 1e30
    got, _ = check(M, l, None, 4, {**BASE, "sigmoid": False}, 1, 64, exact=True)
    assert np.isfinite(got["topk_w"]).all()


def test_plain_softmax_gate_is_moe_route(M):
    """Without groups, bias or scale, a renormalised softmax is moe_route, to the whole number."""
    l = np.random.default_rng(5).standard_normal((1500, 256)).astype(np.float32)
    got = route(M, l, None, 8, {**BASE, "sigmoid": False}, 8, 40)
    p = M.problem(1500, 8, 256, 8, 8, 40)
    b = M.alloc_buffers(p, DEV)
    M.moe_route(p, torch.from_numpy(l).to(DEV), b["topk_idx"], b["topk_w"], b["counts"], b["offsets"], b["slot"],
                b["rank_counts"], b["dropped"], b["workspace"])
    torch.cuda.synchronize()
    for n in ("topk_idx", "counts", "offsets", "slot", "rank_counts", "dropped"):
        assert np.array_equal(got[n], b[n].cpu().numpy()), n
    assert np.allclose(got["topk_w"], b["topk_w"].cpu().numpy(), rtol=2.0 ** -20)


def test_empty_batch_writes_zero_counts(M):
    got = route(M, np.zeros((0, 64), np.float32), None, 4, BASE, 4, 8)
    for n in ("counts", "offsets", "rank_counts", "dropped"):
        assert (got[n] == 0).all(), n


def test_another_stream_and_repeats_give_the_same_bits(M):
    l = np.random.default_rng(6).standard_normal((777, 160)).astype(np.float32)
    c = {**BASE, "G": 8, "top_g": 3, "sigmoid": False, "renorm": False}
    a = route(M, l, None, 6, c, 8, 20)
    s = torch.cuda.Stream()
    for _ in range(3):
        b = route(M, l, None, 6, c, 8, 20, stream=s)
        for n in a:
            assert a[n].tobytes() == b[n].tobytes(), n


# ---- gradient ----

def backward(M, l, idx, w, d_w, c, bf16, with_logits=True):
    T, E = l.shape
    p = M.problem(T, 8, E, idx.shape[1], 1, 4)
    x = on_device(l, bf16)
    d = torch.full_like(x, 7.0)
    M.moe_route_gated_backward(p, gate_of(M, c, bf16), x if with_logits else None,
                               torch.from_numpy(idx).to(DEV), torch.from_numpy(w).to(DEV),
                               torch.from_numpy(d_w).to(DEV), d)
    torch.cuda.synchronize()
    return d.float().cpu().numpy()


def check_backward(M, l, bias, k, c, bf16, seed):
    l = P.bf16_round(l) if bf16 else np.asarray(l, np.float32)
    fwd = route(M, l, bias, k, c, bf16=bf16)
    d_w = np.random.default_rng(seed).standard_normal(fwd["topk_w"].shape).astype(np.float32)
    ok = fwd["slot"] >= 0
    d_w[~ok] = np.nan                                   # what stands at no pair is not used
    got = backward(M, l, fwd["topk_idx"], fwd["topk_w"], d_w, c, bf16)
    ref, mag = P.gate_backward(l, fwd["topk_idx"], ok, d_w, c["sigmoid"], c["renorm"], c["scale"])
    bar = (48 + l.shape[1] / 32) * 2.0 ** -24 * mag + (2.0 ** -8 * np.abs(ref) if bf16 else 0) + 1e-37
    assert (np.abs(got - ref) <= bar).all(), (np.abs(got - ref) / bar).max()
    return fwd, d_w, ok, ref


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("shape", [(1, 256, 8), (37, 64, 6), (300, 6, 3), (5, 1003, 16), (9, 1, 1), (1111, 160, 6),
                                   (3, 8, 8), (17, 1024, 2)])
def test_backward(M, shape, renorm, sigmoid, bf16):
    T, E, k = shape
    rng = np.random.default_rng(E)
    check_backward(M, 2 * rng.standard_normal((T, E)), None, k,
                   {**BASE, "sigmoid": sigmoid, "renorm": renorm, "scale": 2.5}, bf16, E + 1)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_backward_against_differences(M, renorm, sigmoid):
    """The 64-bit formula, which the kernel is held to, against central differences of the weights themselves
    (step 1e-5: the second-order error is under 1e-9 of the weights' scale, rounding 1e-11)."""
    rng = np.random.default_rng(8)
    c = {**BASE, "G": 4, "top_g": 2, "sigmoid": sigmoid, "renorm": renorm, "scale": 2.5}
    l = rng.standard_normal((12, 24)).astype(np.float32)
    fwd, d_w, ok, ref = check_backward(M, l, 0.1 * rng.standard_normal(24), 5, c, False, 9)
    got = backward(M, l, fwd["topk_idx"], fwd["topk_w"], d_w, c, False)
    for t in range(12):
        for e in range(24):
            up, down = l[t].astype(np.float64), l[t].astype(np.float64)
            up[e] += 1e-5
            down[e] -= 1e-5
            f = [P.weights_of(v, fwd["topk_idx"][t], ok[t], sigmoid, renorm, 2.5) for v in (up, down)]
            assert abs(((f[0] - f[1]) * d_w[t]).sum() / 2e-5 - ref[t, e]) < 1e-7
            assert abs(((f[0] - f[1]) * d_w[t]).sum() / 2e-5 - got[t, e]) < 1e-5


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_backward_of_masked_rows_is_zero(M, renorm, sigmoid):
    rng = np.random.default_rng(10)
    l = rng.standard_normal((50, 40))
    l[rng.random(l.shape) < 0.9] = -np.inf
    l[3] = np.nan
    l[4] = LOW_F32
    check_backward(M, l, None, 6, {**BASE, "sigmoid": sigmoid, "renorm": renorm}, False, 11)


def test_backward_of_a_renormalised_softmax_needs_no_logits(M):
    l = np.random.default_rng(12).standard_normal((60, 64)).astype(np.float32)
    c = {**BASE, "sigmoid": False}
    fwd, d_w, _, _ = check_backward(M, l, None, 6, c, False, 13)
    a = backward(M, l, fwd["topk_idx"], fwd["topk_w"], d_w, c, False)
    b = backward(M, l, fwd["topk_idx"], fwd["topk_w"], d_w, c, False, with_logits=False)
    assert np.array_equal(a, b)


def test_backward_of_very_low_logits(M):
    """Sigmoids that underflow: the renormalised weights, and so their gradient, are those of a softmax."""
    l = np.random.default_rng(14).standard_normal((40, 24)) - np.linspace(0, 300, 40)[:, None]
    for renorm in (True, False):
        check_backward(M, l, None, 5, {**BASE, "renorm": renorm, "G": 4, "top_g": 2}, False, 15)
