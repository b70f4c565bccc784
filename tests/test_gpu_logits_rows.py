"""sv_adjust_logits where a row of more than 4096 ids is one workgroup's: from 8192 rows on (fewer
rows are cut into parts of 2049 .. 4096 ids).  Out of place and in place, against the fp64
oracle; tolerances as in test_gpu_logits.py."""

import pytest
import torch

from test_gpu_logits import Case

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("dtype,vocab", [(BF, 5001), (F32, 4100)])
@pytest.mark.parametrize("cap", [None, 3])
def test_rows_of_one_workgroup(dtype, vocab, cap):
    """An odd last tile; with a list of every id said and with one that does not hold them."""
    c = Case(71, 2050, 3, vocab, dtype, said=12, bias=3, cap=cap)
    assert c.z.shape[0] >= 8192
    c.check()
