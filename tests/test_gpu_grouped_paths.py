"""Paths through the grouped kernels that the layouts of test_gpu_grouped.py do not take."""
import pytest

from test_gpu_grouped import Case, check_dw, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts,K,N", [
    ([64, 128, 64, 0, 192, 64, 320, 64, 64, 128] * 4, 1024, 1024),  # several items per block
    ([64, 192, 128, 64, 256, 64, 0, 128, 64], 1032, 1024),          # the same on smaller tiles
    ([64, 63, 64, 65, 128, 1, 64, 127] * 3, 1032, 520)])            # whole and partial last stages
def test_gathered_weight_gradients_of_whole_stages(counts, K, N):
    """Experts whose rows are a multiple of a stage: the copies go from one item's last whole
    stage straight on to the next item's token list."""
    say(f"case {counts[:10]} K={K} N={N}")
    c = Case(counts, K, N, extra=3, tokens=301, seed=len(counts))
    check_dw(c, bias=True)
    check_dw(c, accumulate=True)
