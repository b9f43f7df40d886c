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
