"""moe_route around the batch sizes at which its finaliser changes: as many tiles of 32 tokens as SMs and one more, and
a third more than SMs past 512 experts. Whole numbers, so equal to a plain count."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def M():
    from combine_router_top_gb300 import build as B
    B.build()
    import combine_router_top_gb300 as M
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return M


@pytest.mark.parametrize("E,k,R", [(8, 2, 4), (256, 8, 8), (513, 3, 27), (1024, 16, 8)])
@pytest.mark.parametrize("more", [-5, 0, 1, 40])
def test_slots_and_totals(M, E, k, R, more):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tiles = sms + sms // 3 if E > 512 else sms
    T = 32 * tiles + more
    C = max(1, T * k // E)                              # about half of the experts overflow
    rng = np.random.default_rng(E + more)
    logits = rng.integers(0, 200, (T, E)).astype(np.float32)         # with ties
    p = M.problem(T, 8, E, k, R, C)
    b = M.alloc_buffers(p, DEV)
    b["workspace"].fill_(0x55)
    M.moe_route(p, torch.from_numpy(logits).to(DEV), b["topk_idx"], b["topk_w"], b["counts"], b["offsets"], b["slot"],
                b["rank_counts"], b["dropped"], b["workspace"])
    torch.cuda.synchronize()
    got = {n: b[n].cpu().numpy() for n in ("topk_idx", "counts", "offsets", "slot", "rank_counts", "dropped")}
    idx = np.argsort(-logits, axis=1, kind="stable")[:, :k]
    assert np.array_equal(got["topk_idx"], idx)
    flat = idx.ravel()                                  # a token's experts differ: pairs count as tokens do
    order = np.argsort(flat, kind="stable")
    counts = np.bincount(flat, minlength=E)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    slot = np.empty(flat.size, np.int64)
    slot[order] = np.arange(flat.size) - offsets[flat[order]]
    kept = np.minimum(counts, C)
    assert np.array_equal(got["counts"], counts) and np.array_equal(got["offsets"], offsets)
    assert np.array_equal(got["slot"].ravel(), np.where(slot < C, slot, -1))
    assert np.array_equal(got["rank_counts"], kept.reshape(R, -1).sum(1))
    assert got["dropped"][0] == (counts - kept).sum()
