"""sv_latent_attend under very small scales, where a first tile that holds no position must
not be taken for one whose scores are near the rest: tolerances as in test_gpu_latent.py.

32 / scale, the distance in products at which sums start again from larger maxima, passes
fp32's range for scales below 9.4e-38."""

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


@pytest.mark.parametrize("scale", [1e-30, 5e-38, -5e-38, 1e-38])
@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("heads,k_max,parts", [(128, 64, 1), (5, None, 2)])
def test_scales_near_zero_behind_missing_pages(scale, dtype, heads, k_max, parts):
    """The first pages are missing: every weight is the same, those of the absent ones 0."""
    b = Batch(31, [2, 1], [90, 40], heads, 512, 16, dtype, k_max=k_max)
    b.scale = scale
    b.table[0, :2], b.table[1, :2] = -1, b.kv.shape[0]
    ws = sv.sv_latent_attend_workspace_bytes(b.n, b.k_max, heads, 512, b.table.shape[1], 16)
    assert ws == (parts > 1) * parts * b.n * (b.k_max + 1) * heads * (512 + 2) * 4
    b.device().check(want_err=sv.SV_DEV_BAD_PAGE)
