"""sv_cache_attend_shared with offsets that differ from those the batch was made with and are valid
all the same: against the fp64 oracle, nothing reported.  Tolerances as in test_gpu_shared.py."""

import pytest
import torch

from test_gpu_shared import BF, F8, Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("cu", [[0, 2, 2, 4, 6], [0, 0, 1, 4, 6], [0, 2, 4, 4, 4], [0, 0, 0, 3, 6]])
def test_rows_moved_between_groups(dtype, cu):
    """Requests, and a whole group, without rows; others with more than they had."""
    b = Batch(20, [(48, [(2, 13), (1, 20)]), (20, [(1, 4), (2, 5)])], 4, 2, 64, 16, dtype, k_max=2)
    b.cu = torch.tensor(cu, dtype=torch.int32)
    b.device().check()
