"""The combine's gradient for batches past two tokens to an SM with rows of more than 1024 elements, whose blocks are of
7 and of 8 warps, against the formula with the inputs and the bars of test_gpu_combine_backward."""
import numpy as np
import pytest
import torch

from test_gpu_combine_backward import DEV, M, inputs, run  # noqa: F401  (M is a fixture)

pytestmark = pytest.mark.gpu

# elements of a row: warps to a block. A turn is 224 or 256 chunks of 8: 7 warps for one turn (193 and 224 chunks), two
# (440) and three (513), 8 warps for one (242 and 256) and two (449)
WIDTHS = {1544: 7, 1792: 7, 3520: 7, 4104: 7, 1936: 8, 2048: 8, 3592: 8}


@pytest.mark.parametrize("k", [2, 6, 16])
@pytest.mark.parametrize("H", WIDTHS)
def test_against_the_formula(M, H, k):  # noqa: F811
    chunks = H // 8
    assert (7 if -(-chunks // 224) * 224 < -(-chunks // 256) * 256 else 8) == WIDTHS[H]
    T, E, C = 3 * torch.cuda.get_device_properties(0).multi_processor_count + 1, 20, 40 * k
    idx, slot, w, _, _ = inputs(T, 8, E, k, C, H + k, drop=0.1)
    g = torch.Generator(device=DEV).manual_seed(H + k)
    y = torch.randn((E, C, H), device=DEV, generator=g).to(torch.bfloat16)
    d_out = torch.randn((T, H), device=DEV, generator=g).to(torch.bfloat16)
    up = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    p = M.problem(T, H, E, k, 1, C)
    d_y, d_w = torch.full_like(y, 3.0), torch.full((T, k), 7.0, device=DEV)
    M.moe_combine_backward(p, y, d_out, up(idx), up(w), up(slot), d_y, d_w)
    torch.cuda.synchronize()
    ref, ref_w, mag = torch.full_like(y, 3.0), np.zeros((T, k)), np.zeros((T, k))
    for j in range(k):
        t = np.nonzero(slot[:, j] >= 0)[0]
        e, s = idx[t, j], slot[t, j]
        rows = d_out[up(t)]
        ref[up(e).long(), up(s).long()] = (up(w[t, j])[:, None] * rows.float()).to(torch.bfloat16)
        prod = y[up(e).long(), up(s).long()].double() * rows.double()
        ref_w[t, j], mag[t, j] = prod.sum(1).cpu().numpy(), prod.abs().sum(1).cpu().numpy()
    assert 0 < (slot < 0).sum() < slot.size
    assert torch.equal(d_y.view(torch.int16), ref.view(torch.int16))
    assert (np.abs(d_w.cpu().numpy() - ref_w) <= (H / 32 + 80) * 2.0 ** -24 * mag).all()


@pytest.mark.parametrize("H", [3520, 3592])
def test_the_grid_and_the_stream_change_no_bit(M, H):  # noqa: F811
    T = 3 * torch.cuda.get_device_properties(0).multi_processor_count + 1
    a = inputs(T, H, 8, 2, 100, 3, drop=0.1)
    d_y, d_w = run(M, *a)
    for max_blocks in (1, 7, 200, 100000):
        b_y, b_w = run(M, *a, max_blocks=max_blocks, stream=torch.cuda.Stream())
        assert np.array_equal(d_y, b_y) and np.array_equal(d_w, b_w)
