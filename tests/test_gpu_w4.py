"""The experts' 4-bit products on the GPU against a plain form in 64 bits.

Tolerance. With S = sum of |x| |q - 8| scale over a row's inputs: an MMA step of 16 inputs rounds its sum and its add
into the accumulator (2), at most K/16 steps; a group's sum is scaled and added once (2 for each of K/32 groups at
most, 1 more for an fp8 row's block scale), and at most 32 partial sums are joined: every rounding is at most 2^-24 of
S, so |r - r64| <= (K/8 + K/16 + 32) 2^-24 S =: B. With the gate, silu moves by at most 1.1 of its argument's error and
is formed in 4 more roundings: 1.1 B_g |u| + |silu(g)| B_u + B_g B_u + 2^-21 |y|. One rounding to bf16: 2^-8 of the
value (half an ulp is at most 2^-9 of it, doubled for the step across a binade) and 2^-133 at the lowest values."""
import numpy as np
import pytest
import torch

import plain64 as P

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SENTINEL = 3.0


@pytest.fixture(scope="module")
def M():
    from combine_router_top_gb300 import build as B
    B.build()
    import combine_router_top_gb300 as M
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return M


def make(M, counts, C, K, N, group, gate, fp8, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    E, rows = len(counts), 2 * N if gate else N
    x = torch.randn((E, C, K), device=DEV, generator=g)
    if fp8:
        b = x.unflatten(-1, (-1, 128))
        s = b.abs().amax(-1) / 448.0
        x, s = (b / s[..., None]).flatten(-2).to(torch.float8_e4m3fn).view(torch.uint8), s
    else:
        x, s = x.to(torch.bfloat16), None
    for e, n in enumerate(counts):                      # rows past the count are no inputs
        if n < C:
            if fp8:
                x[e, max(n, 0):], s[e, max(n, 0):] = 0x7F, float("nan")
            else:
                x[e, max(n, 0):] = float("nan")
    codes = torch.randint(0, 16, (E, rows, K), dtype=torch.uint8, device=DEV, generator=g)
    scale = (torch.randn((E, rows, K // group), device=DEV, generator=g) * 0.1).to(torch.bfloat16)
    return x, s, codes, M.w4_pack(codes), scale


def run(M, counts, x, s, w_q, scale, N, group, gate, T=None, max_blocks=0, stream=None):
    E, C, K = x.shape
    T = max(1, min(max(counts), 1 << 20)) if T is None else T
    p = M.problem(T, 8 if s is None else 128, E, min(E, 4), 1, C, 0 if s is None else 1, max_blocks)
    w = M.w4(K, N, group, M.MOE_ACT_SILU_GATE if gate else M.MOE_ACT_NONE)
    y = torch.full((E, C, N), SENTINEL, dtype=torch.bfloat16, device=DEV)
    ws = torch.full((M.moe_expert_w4_workspace_bytes(p, w),), 0x55, dtype=torch.uint8, device=DEV)
    c = torch.tensor(counts, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()                            # the inputs are made on the default stream
    M.moe_expert_w4(p, w, x, s, c, w_q, scale, y, ws, stream=stream)
    torch.cuda.synchronize()
    assert M.moe_device_status() == M.MOE_OK
    return y


def check(M, counts, C, K, N, group, gate, fp8, seed=0, T=None, max_blocks=0):
    x, s, codes, w_q, scale = make(M, counts, C, K, N, group, gate, fp8, seed)
    y = run(M, counts, x, s, w_q, scale, N, group, gate, T, max_blocks).double().cpu().numpy()
    for e, n in enumerate(counts):
        n = min(n, C)
        assert (y[e, n:] == SENTINEL).all()
        if n == 0:
            continue
        v = x[e, :n].view(torch.float8_e4m3fn).double() * s[e, :n].double().repeat_interleave(128, 1) if fp8 \
            else x[e, :n].double()
        r, S = P.w4_rows(v.cpu().numpy(), codes[e].cpu().numpy(), scale[e].double().cpu().numpy(), group)
        B = (K / 8 + K / 16 + 32) * 2.0 ** -24 * S
        if gate:
            g, u = r[:, :N], r[:, N:]
            ref = P.silu(g) * u
            B = 1.1 * B[:, :N] * np.abs(u) + np.abs(P.silu(g)) * B[:, N:] + B[:, :N] * B[:, N:] + 2.0 ** -21 * np.abs(ref)
        else:
            ref = r
        err = np.abs(y[e, :n] - ref)
        bar = B + 2.0 ** -8 * np.abs(ref) + 2.0 ** -133
        assert (err <= bar).all(), (e, (err / bar).max())


SHAPES = [
    # counts, C, K, N
    ([1], 1, 128, 8),
    ([1], 4, 256, 24),
    ([3, 0, 1], 3, 384, 16),
    ([0, 8, 9, 7], 12, 1408, 40),
    ([16, 17, 2, 0, 15], 17, 512, 136),
    ([5, 40, 3], 32, 640, 128),                         # one expert past its capacity
    ([33, 1, 64], 64, 1152, 264),
    ([130, 0, 100, 257], 257, 256, 264),
    ([1, 0, 0, 0, 0, 0, 0, 2], 2, 7168, 72),
]


def test_the_layout_is_the_stated_one(M):
    codes = torch.randint(0, 16, (3, 5, 384), dtype=torch.uint8)
    packed = M.w4_pack(codes)
    assert np.array_equal(P.w4_codes(packed.numpy(), 384), codes.numpy())
    assert torch.equal(M.w4_unpack(packed), codes)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_rows(M, shape, group, gate, fp8):
    counts, C, K, N = SHAPES[shape]
    check(M, counts, C, K, N, group, gate, fp8, 10 * shape)


@pytest.mark.parametrize("T", [4, 60, 4096])
@pytest.mark.parametrize("fp8", [False, True])
def test_the_batch_that_the_problem_states_changes_no_result_past_rounding(M, T, fp8):
    """Few or many tokens choose how the work is split; the rows are what counts says."""
    check(M, [7, 0, 4, 30], 48, 896, 152, 64, True, fp8, 5, T=T)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_long_rows_and_many_tiles_to_a_block(M, group, fp8):
    """29 blocks of inputs (an odd number, over the rings' depths) and nine or more tiles of 1 to 64 rows for each of two
    thread blocks: what is counted per block, tile and use goes around several times."""
    check(M, [20, 33, 5, 64, 1, 0, 17, 100], 100, 3712, 264, group, True, fp8, 6, T=4096, max_blocks=2)


@pytest.mark.parametrize("gate", [False, True])
def test_no_rows_at_all(M, gate):
    check(M, [0, 0, 0], 8, 256, 16, 64, gate, False)


@pytest.mark.parametrize("T", [8, 4096])
@pytest.mark.parametrize("max_blocks", [1, 5, 1000])
def test_the_grid_and_the_stream_change_no_bit(M, max_blocks, T):
    counts = [20, 1, 0, 70]
    x, s, _, w_q, scale = make(M, counts, 70, 768, 200, 64, True, False, 1)
    a = run(M, counts, x, s, w_q, scale, 200, 64, True, T)
    for st in (None, torch.cuda.Stream()):
        assert torch.equal(a, run(M, counts, x, s, w_q, scale, 200, 64, True, T, max_blocks, st))


def test_nan_and_infinity_stay_in_their_rows(M):
    counts = [9, 20]
    x, s, _, w_q, scale = make(M, counts, 20, 256, 48, 128, False, False, 2)
    a = run(M, counts, x, s, w_q, scale, 48, 128, False)
    x[0, 3, 5], x[1, 19, 200] = float("nan"), float("inf")
    b = run(M, counts, x, s, w_q, scale, 48, 128, False)
    bad = ~torch.isfinite(b.float())
    assert bad[0, 3].all() and bad[1, 19].all() and int(bad.any(2).sum()) == 2
    keep = ~bad
    assert torch.equal(a[keep], b[keep])


@pytest.mark.parametrize("T", [8, 4096])
def test_matrices_past_four_gigabytes(M, T):
    """The last expert of 5.9 GB of weights and of 4.3 GB of rows: offsets that pass 32 bits."""
    E, K, N, C = 200, 7168, 8192, 1500
    w_q = torch.zeros((E, N, K // 2), dtype=torch.uint8, device=DEV)
    scale = torch.ones((E, N, K // 128), dtype=torch.bfloat16, device=DEV)
    x = torch.zeros((E, C, K), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(3)
    codes = torch.randint(0, 16, (N, K), dtype=torch.uint8, device=DEV, generator=g)
    w_q[E - 1] = M.w4_pack(codes)
    x[E - 1] = torch.randn((C, K), device=DEV, generator=g)
    counts = [0] * (E - 1) + [C]
    y = run(M, counts, x, None, w_q, scale, N, 128, False, T=T)
    for r in (0, C - 1):
        ref = x[E - 1, r].double() @ (codes.double() - 8.0).T
        S = x[E - 1, r].double().abs() @ (codes.double() - 8.0).abs().T
        bar = (K / 8 + K / 16 + 32) * 2.0 ** -24 * S + 2.0 ** -8 * ref.abs()
        assert ((y[E - 1, r].double() - ref).abs() <= bar).all()
    assert (y[: E - 1] == SENTINEL).all()
