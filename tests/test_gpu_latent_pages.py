"""A page that is not there is reported by sv_latent_attend wherever it lies, alone."""

import pytest
import torch

import adaptive_draft_verification_amd as sv
from test_gpu_latent import Batch

pytestmark = pytest.mark.gpu

BF, F8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("page,missing", [(16, p) for p in range(8)] + [(1, p) for p in (1, 63, 64, 99)])
def test_one_missing_page_is_reported(dtype, page, missing):
    b = Batch(51, [2, 1], [120, 50], 5, 256, page, dtype)
    b.table[0, missing] = -1 if missing % 2 else b.kv.shape[0]
    b.device().check(want_err=sv.SV_DEV_BAD_PAGE)
