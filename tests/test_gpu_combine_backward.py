"""The combine's gradient on the GPU against its formula in 64 bits.

d_y is one fp32 product rounded to bf16: bit for bit. d_topk_w sums H exact products in fp32: a lane's chain is at
most H/32 + 64 long, then 5 steps over the warp and 4 over warps, so its error is at most (H/32 + 80) 2^-24 of the
sum of the products' magnitudes."""
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


def inputs(T, H, E, k, C, seed, drop=0.0):
    rng = np.random.default_rng(seed)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ok = rng.random((T, k)) >= drop
    slot = P.count(idx, ok, E, 1, C)["slot"]
    w = rng.standard_normal((T, k)).astype(np.float32)
    return idx, slot, w, P.bf16_round(rng.standard_normal((E, C, H))), P.bf16_round(rng.standard_normal((T, H)))


def run(M, idx, slot, w, y, d_out, max_blocks=0, stream=None):
    T, k = idx.shape
    E, C, H = y.shape
    p = M.problem(T, H, E, k, 1, C, 0, max_blocks)
    d_y = torch.full((E, C, H), 3.0, dtype=torch.bfloat16, device=DEV)
    d_w = torch.full((T, k), 7.0, device=DEV)
    up = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    ins = up(y).to(torch.bfloat16), up(d_out).to(torch.bfloat16), up(idx), up(w), up(slot)
    torch.cuda.synchronize()                            # the inputs are made on the default stream
    M.moe_combine_backward(p, *ins, d_y, d_w, stream=stream)
    torch.cuda.synchronize()
    return d_y.float().cpu().numpy(), d_w.cpu().numpy()


def check(M, idx, slot, w, y, d_out, **kw):
    d_y, d_w = run(M, idx, slot, w, y, d_out, **kw)
    H = y.shape[2]
    ref = np.full_like(d_y, 3.0)                        # rows of no pair are left as they were
    for t, j in np.ndindex(idx.shape):
        e, s = idx[t, j], slot[t, j]
        if s < 0:
            assert d_w[t, j] == 0.0
            continue
        ref[e, s] = P.bf16_round(w[t, j] * d_out[t])
        prod = y[e, s].astype(np.float64) * d_out[t]
        assert abs(d_w[t, j] - prod.sum()) <= (H / 32 + 80) * 2.0 ** -24 * np.abs(prod).sum()
    assert np.array_equal(d_y, ref)
    return d_y, d_w


@pytest.mark.parametrize("T,H,E,k,C", [
    (1, 8, 1, 1, 1), (1, 7168, 16, 8, 1), (5, 512, 4, 2, 3), (9, 520, 8, 6, 9), (33, 1032, 8, 3, 20),
    (6, 2056, 16, 16, 6), (7, 4096, 4, 4, 7), (3, 16384, 4, 2, 3), (2, 65536, 3, 3, 2), (64, 256, 32, 9, 8),
    (11, 1024, 8, 8, 11), (40, 2048, 8, 2, 20), (700, 64, 8, 2, 300), (13, 1792, 8, 5, 9)])
def test_against_the_formula(M, T, H, E, k, C):
    check(M, *inputs(T, H, E, k, C, T + H + E))


def test_dropped_pairs_and_tokens_without_any(M):
    a = inputs(60, 264, 8, 4, 6, 1, drop=0.3)
    a[1][5] = -1
    check(M, *a)


def test_nan_and_infinity_stay_in_their_pairs(M):
    idx, slot, w, y, d_out = inputs(20, 128, 8, 2, 20, 2)
    y[idx[3, 1], slot[3, 1]] = np.nan                   # poisons d_w[3][1] alone
    d_out[4, 7] = np.inf
    d_y, d_w = run(M, idx, slot, w, y, d_out)
    bad = ~np.isfinite(d_w)
    assert bad[3, 1] and bad[4].all() and bad.sum() == 3
    row = np.zeros(y.shape[:2], bool)
    row[idx[4], slot[4]] = True
    assert (~np.isfinite(d_y)).any(2).sum() == 2 and (~np.isfinite(d_y)).any(2)[row].all()


@pytest.mark.parametrize("max_blocks", [1, 7, 1000])
def test_the_grid_and_the_stream_change_no_bit(M, max_blocks):
    a = inputs(90, 2304, 8, 3, 40, 3)
    d_y, d_w = run(M, *a)
    for s in (None, torch.cuda.Stream()):
        b_y, b_w = run(M, *a, max_blocks=max_blocks, stream=s)
        assert np.array_equal(d_y, b_y) and np.array_equal(d_w, b_w)


def test_against_differences_of_the_combine(M):
    """<d_out, combine(y, w)> moves with w and with y as the gradients say: the sum is linear in each, so one step of
    1 in float64 gives the slope itself (to the rounding of d_y to bf16 and of the sums)."""
    idx, slot, w, y, d_out = inputs(10, 64, 6, 3, 6, 4)
    d_y, d_w = run(M, idx, slot, w, y, d_out)

    def loss(y, w):
        out = np.zeros(d_out.shape)
        for t, j in np.ndindex(idx.shape):
            if slot[t, j] >= 0:
                out[t] += w[t, j] * y[idx[t, j], slot[t, j]]
        return (out * d_out).sum()
    y, w = y.astype(np.float64), w.astype(np.float64)
    for t, j in [(0, 0), (3, 2), (9, 1)]:
        if slot[t, j] < 0:
            continue
        w2, y2 = w.copy(), y.copy()
        w2[t, j] += 1.0
        assert abs(loss(y, w2) - loss(y, w) - d_w[t, j]) < 1e-4
        y2[idx[t, j], slot[t, j], 11] += 1.0
        assert abs(loss(y2, w) - loss(y, w) - d_y[idx[t, j], slot[t, j], 11]) < 2.0 ** -8 * abs(w[t, j] * d_out[t, 11]) + 1e-10


def test_rows_past_four_gigabytes(M):
    """Row offsets that pass 32 bits in bytes and in elements: one row at the end of a 5 GB buffer."""
    E, C, H = 320, 1024, 8192
    y = torch.zeros((E, C, H), dtype=torch.bfloat16, device=DEV)
    d_y = torch.zeros_like(y)
    g = torch.randn((1, H), device=DEV).to(torch.bfloat16)
    y[E - 1, C - 1] = torch.randn(H, device=DEV)
    p = M.problem(1, H, E, 1, 1, C)
    i = torch.tensor([[E - 1]], dtype=torch.int32, device=DEV)
    s = torch.tensor([[C - 1]], dtype=torch.int32, device=DEV)
    d_w = torch.empty((1, 1), device=DEV)
    M.moe_combine_backward(p, y, g, i, torch.full((1, 1), 0.5, device=DEV), s, d_y, d_w)
    torch.cuda.synchronize()
    assert torch.equal(d_y[E - 1, C - 1], (0.5 * g[0].float()).to(torch.bfloat16))
    ref = (y[E - 1, C - 1].double() * g[0].double()).sum().item()
    assert abs(d_w.item() - ref) < 1e-3
    assert not d_y[: E - 1].any() and not d_y[E - 1, : C - 1].any()
