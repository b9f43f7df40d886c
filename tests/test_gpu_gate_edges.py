"""The gated route and its gradient at the ends of their ranges, against the plain form in 64 bits.

Weights of a renormalised sigmoid: a score takes exp (2 ulp, twice, the second at most halved), a sum and a division, 8
roundings of 2^-24; the sum over the choices the same and 5 more, the quotient and the scale 2: 23 x 2^-24, under 2^-19.
Gradients: the bar of test_gpu_gate."""
import numpy as np
import pytest
import torch

import plain64 as P
from test_gpu_gate import BASE, DEV, M, backward, check_backward, route  # noqa: F401  (M is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("top", [3.0, 0.25, 0.0, -0.5, -7.0, -29.0, -29.99, -30.0, -31.5, -88.0, -1000.25])
@pytest.mark.parametrize("below", [2.0, 40.0, 66.0, 80.0])
def test_renormalised_sigmoids_far_below_the_best(M, top, below):  # noqa: F811
    """The quotient of a choice e^-below under the row's best is that, although its own sigmoid may be 0 in fp32."""
    rng = np.random.default_rng(int(below))
    l = (top - below * rng.random((50, 16))).astype(np.float32)
    l[:, 5], l[:, 11] = top, top - below
    c = {**BASE, "scale": 2.5}
    got = route(M, l, None, 16, c)
    idx, ok, w, _ = P.gate(l, None, 16, **c)
    assert ok.all() and np.array_equal(got["topk_idx"], idx)
    assert (np.abs(got["topk_w"] - w) <= 2.0 ** -19 * w).all(), np.abs(got["topk_w"] / w - 1).max()
    fwd, _, ok, ref = check_backward(M, l, None, 16, c, False, 3)
    assert (fwd["topk_w"] > 0).all() and (ref != 0).all()


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E", [24, 27])
@pytest.mark.parametrize("scale", [1e-30, 1e-38, -1.1e-39, 1e-44, 1e30, -3e38])
def test_gradients_at_scales_of_any_size(M, scale, E, renorm, sigmoid):  # noqa: F811
    """Every finite scale but 0 has finite gradients. Below 2^-126 the weights themselves are held to 2^-149, which moves
    dot by that over the scale: the bar takes one such step of each weight, for the gradient and for dot."""
    rng = np.random.default_rng(5)
    T, k = 60, 5
    l = rng.standard_normal((T, E)).astype(np.float32)
    scale = float(np.float32(scale))
    c = {**BASE, "sigmoid": sigmoid, "renorm": renorm, "scale": scale}
    fwd = route(M, l, None, k, c)
    d_w = (0.1 * rng.standard_normal((T, k))).astype(np.float32)
    got = backward(M, l, fwd["topk_idx"], fwd["topk_w"], d_w, c, False)
    ref, mag = P.gate_backward(l, fwd["topk_idx"], np.ones((T, k), bool), d_w, sigmoid, renorm, scale)
    step = 2.0 ** -149 * np.abs(d_w).sum(1)[:, None] * 2 + 4 * 2.0 ** -149
    assert (np.abs(got - ref) <= (48 + E / 32) * 2.0 ** -24 * mag + step).all(), np.abs(got - ref).max()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("E", [24, 27])
@pytest.mark.parametrize("left", [21, 3])
def test_an_expert_that_only_the_bias_masks_stays_in_the_softmax(M, left, E, bf16):  # noqa: F811
    """Weights s_e over all experts: a bias of -inf takes an expert out of the choice, not out of the sum, so its logit has
    a gradient. Against the formula, and against central differences of the weights (second order under 1e-9, fp32 and
    bf16 roundings of the gradient by the formula's bar). With 3 experts left of k = 5 the last choices are no pairs."""
    rng = np.random.default_rng(left)
    bias = 0.1 * rng.standard_normal(E)
    masked = rng.permutation(E)[:E - left]
    bias[masked] = -np.inf
    c = {**BASE, "sigmoid": False, "renorm": False, "scale": 2.5}
    l = rng.standard_normal((20, E)).astype(np.float32)
    l[:, masked[0]] = 4.0                               # the largest score of all
    l[3, masked[0]] = -np.inf                           # masked both ways
    fwd, d_w, ok, ref = check_backward(M, l, bias, 5, c, bf16, 4)
    assert (ok.sum(1) == min(left, 5)).all() and not np.isin(fwd["topk_idx"][ok], masked).any()
    assert ref[3, masked[0]] == 0 and (ref[:3, masked[0]] != 0).all()
    x = P.bf16_round(l) if bf16 else l
    for t, e in [(0, masked[0]), (5, masked[-1]), (7, fwd["topk_idx"][7, 0])]:
        f = []
        for s in (1e-5, -1e-5):
            v = x[t].astype(np.float64)
            v[e] += s
            f.append(P.weights_of(v, fwd["topk_idx"][t], ok[t], False, False, 2.5))
        slope = ((f[0] - f[1])[ok[t]] * d_w[t][ok[t]]).sum() / 2e-5
        assert abs(slope - ref[t, e]) < 1e-7


@pytest.mark.parametrize("T,E,k,C", [(1, 16, 4, 4), (70, 16, 4, 12), (500, 64, 8, 40)])
def test_the_gradient_of_a_bf16_dispatch_is_the_combine_with_weights_of_one(M, T, E, k, C):  # noqa: F811
    """x[t] is copied to the rows of its kept pairs, so its gradient is the sum of those rows' gradients: at most k fp32
    roundings of the magnitudes and one to bf16 (half an ulp, doubled across a binade). Checked against <d_rows, rows>,
    linear in x, too: a step of 1 in an element of x moves it by the element's exact gradient."""
    H = 136
    torch.manual_seed(T)
    rng = np.random.default_rng(T)
    l = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(DEV)
    p = M.problem(T, H, E, k, 1, C)
    b = M.alloc_buffers(p, DEV)
    x = torch.randn((T, H), device=DEV).to(torch.bfloat16)
    M.moe_route_gated(p, M.gate(), l, None, b["topk_idx"], b["topk_w"], b["counts"], b["offsets"], b["slot"],
                      b["rank_counts"], b["dropped"], b["workspace"])
    d_rows = torch.randn((E, C, H), device=DEV).to(torch.bfloat16)
    d_x = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    M.moe_combine(p, d_rows, b["topk_idx"], torch.ones((T, k), device=DEV), b["slot"], d_x)

    def rows_of(x):
        b["recv"].zero_()
        M.moe_dispatch(p, x, b["topk_idx"], b["slot"], b["recv"], None, b["recv_src"])
        return b["recv"].view(torch.bfloat16).double()
    ref, mag = torch.zeros((T, H), dtype=torch.float64, device=DEV), torch.zeros((T, H), dtype=torch.float64, device=DEV)
    idx, slot = b["topk_idx"].long(), b["slot"].long()
    for j in range(k):
        rows = torch.where((slot[:, j] >= 0)[:, None], d_rows[idx[:, j], slot[:, j].clamp(min=0)].double(), 0.0)
        ref += rows
        mag += rows.abs()
    assert ((d_x.double() - ref).abs() <= k * 2.0 ** -24 * mag + 2.0 ** -8 * ref.abs()).all()
    x[0, 5] = 1.0                                       # exact steps: 1 to 2
    before = rows_of(x)
    x[0, 5] = 2.0
    assert abs(((rows_of(x) - before) * d_rows.double()).sum() - ref[0, 5]) < 1e-12
