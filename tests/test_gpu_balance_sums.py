"""The bias gradient against the 64-bit sum of the gradient rows that the same call
wrote: what the column sums alone are off by."""
import pytest
import torch

from tests._fp8 import U32
from tests._gpu import needs_gpu
from tests.test_gpu_balance import _inputs, _run

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.fixture(scope="module")
def cm():
    import int4_routed_expert_renorm_b200 as m
    return m


def _chain(T):
    """Additions along the longest path of a column sum.  Up to 256 tokens 8 blocks of 16
    warps: a warp's tokens, the block's 16 warps, the 8 blocks.  Above, up to 296 blocks:
    a warp's tokens, 16 warps, the rows of a second-pass warp (every 16th), its 16 warps."""
    if T <= 256:
        return -(-T // 128) + 16 + 8
    blocks = min(-(-T // 16), 296)
    return -(-T // (16 * blocks)) + 16 + -(-blocks // 16) + 16


@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (128, 256, 8), (255, 33, 4), (257, 256, 8), (4736, 64, 4), (4737, 65, 4),
                                   (30011, 256, 8), (9000, 600, 3)])
def test_bias_gradient_is_the_sum_of_the_rows(cm, T, E, k):
    """Each addition is off by half a step of a partial sum, which no sum of magnitudes
    falls short of: chain * 2^-24 * sum |d|."""
    *_, d, db = _run(cm, *_inputs(T, E, k, 3 * T + E, live=0.9))
    assert (db - d.sum(0)).abs().le(_chain(T) * U32 * d.abs().sum(0) + 1e-37).all()
