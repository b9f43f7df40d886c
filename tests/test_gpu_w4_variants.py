"""The variants of the experts' 4-bit products that few sizes reach, against the plain form in 64 bits, with the inputs
and the tolerance of test_gpu_w4."""
import pytest
import torch

from test_gpu_w4 import DEV, M, check, make, run  # noqa: F401  (M is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("blocks", [1, 3, 9, 17, 31])
def test_tiles_with_an_odd_number_of_scales_to_a_row(M, blocks, fp8, gate):  # noqa: F811
    """Groups of 128 over an odd number of input blocks: rows of scales that no 4-byte copy reaches. Three thread blocks
    take ten and more tiles of each width (up to 16, 32 and 64 rows), so that the ring of scales goes around often, and
    the last chunk of 8 groups is filled with 1 or 7."""
    check(M, [64, 3, 30, 0, 17, 100, 16], 100, 128 * blocks, 264, 128, gate, fp8, blocks, T=4096, max_blocks=3)


# The kernel for few rows gives a warp two fragments of matrix rows once live experts x outputs / 16 (32 without the gate)
# reach three to an SM: 8 experts x 1048 / 16 = 524, x 2056 / 32 = 514. Neither size is a multiple of a block's outputs
# (16, or 32), so that the last block's second fragment reads the last matrix row for those past it.
FEW = [1, 0, 3, 2, 8, 1, 2, 3]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("gate,N", [(True, 1048), (True, 2056), (False, 2056)])
@pytest.mark.parametrize("K", [128, 384, 1152])
def test_few_rows_with_two_fragments_to_a_warp(M, K, gate, N, group, fp8):  # noqa: F811
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert len(FEW) * N // (16 if gate else 32) >= 3 * sms
    check(M, FEW, 8, K, N, group, gate, fp8, K + N, T=8)


@pytest.mark.parametrize("gate", [False, True])
def test_few_rows_with_two_fragments_past_the_capacity(M, gate):  # noqa: F811
    """More pairs than rows, several tiles of 8 rows to an expert, and two thread blocks for all of it."""
    check(M, [30, 0, 11, 9, 1, 0, 17, 2], 12, 640, 2056, 64, gate, True, 7, T=7, max_blocks=2)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("gate", [False, True])
def test_the_grid_and_the_stream_change_no_bit_of_two_fragments(M, gate, fp8):  # noqa: F811
    x, s, _, w_q, scale = make(M, FEW, 8, 1152, 2056, 128, gate, fp8, 1)
    a = run(M, FEW, x, s, w_q, scale, 2056, 128, gate, 8)
    for max_blocks in (1, 5, 100000):
        b = run(M, FEW, x, s, w_q, scale, 2056, 128, gate, 8, max_blocks, torch.cuda.Stream())
        assert torch.equal(a, b)
