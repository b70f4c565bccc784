"""Host validation of the latent cache and of attention over shared prefixes (CPU):
refusals come before anything is launched, and the binding refuses what does not fit."""

import ctypes
import math
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from oracle.cache import cache_attend
from oracle.latent import latent_append, latent_attend

sv = pytest.importorskip("adaptive_draft_verification_amd",
                         reason="libspecverify.so not built (python adaptive_draft_verification_amd/build.py)")

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "adaptive_draft_verification_amd", "csrc")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")

FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p(0x1008)


def latent(**kw):
    args = dict(kv=0x1000, dtype=sv.SV_BF16, n_pages=10, page_size=16, latent_dim=512,
                page_stride=16 * 576, token_stride=576, scale=None)
    args.update(kw)
    return ctypes.byref(sv._LatentCache(*args.values()))


def append(c=None, **kw):
    args = dict(table=FAKE, max_pages=4, latent=FAKE, latent_ld=512, rope=FAKE, rope_ld=64,
                row_req=FAKE, row_pos=FAKE, n_rows=4, ctx=FAKE, n_req=2, err=None, stream=None)
    args.update(kw)
    return sv._lib.sv_latent_append(latent() if c is None else c, *args.values())


def attend(c=None, **kw):
    args = dict(table=FAKE, max_pages=4, q=FAKE, q_ld=16 * 576, q_rows=4, n_heads=16, cu=FAKE,
                ctx=FAKE, n_req=2, k_max=3, scale=0.1, out=FAKE, out_ld=16 * 512, lse=None, err=None,
                ws=FAKE, ws_bytes=0, stream=None)
    args.update(kw)
    return sv._lib.sv_latent_attend(latent() if c is None else c, *args.values())


def cache(**kw):
    args = dict(k=0x1000, v=0x1000, dtype=sv.SV_BF16, n_pages=10, page_size=16, n_kv_heads=2,
                head_dim=64, page_stride=16 * 128, token_stride=128, head_stride=64, k_scale=None,
                v_scale=None)
    args.update(kw)
    return ctypes.byref(sv._Cache(*args.values()))


def shared(c=None, **kw):
    args = dict(table=FAKE, max_pages=4, q=FAKE, q_ld=4 * 64, q_rows=4, n_heads=4, cu=FAKE, ctx=FAKE,
                n_req=2, k_max=3, start=FAKE, prefix=FAKE, n_groups=1, scale=0.1, out=FAKE,
                out_ld=4 * 64, lse=None, err=None, ws=FAKE, ws_bytes=0, stream=None)
    args.update(kw)
    return sv._lib.sv_cache_attend_shared(cache() if c is None else c, *args.values())


BAD_LATENT = [dict(latent_dim=128), dict(latent_dim=576), dict(n_pages=-1), dict(page_size=0),
              dict(page_stride=4), dict(token_stride=-8), dict(kv=0x1008),
              dict(dtype=sv.SV_E4M3, token_stride=584), dict(page_stride=2 ** 60)]


@pytest.mark.parametrize("kw", BAD_LATENT)
def test_latent_layouts(kw):
    assert append(latent(**kw)) == attend(latent(**kw)) == sv.SV_ERR_SHAPE


def test_latent_refusals():
    none = ctypes.c_void_p(None)
    assert append(none) == attend(none) == sv.SV_ERR_NULL
    for dtype in (sv.SV_F32, 9):
        assert append(latent(dtype=dtype)) == attend(latent(dtype=dtype)) == sv.SV_ERR_DTYPE
    assert append(latent(kv=None)) == attend(latent(kv=None)) == sv.SV_ERR_NULL
    for name in ("table", "latent", "rope", "row_req", "row_pos", "ctx"):
        assert append(**{name: None}) == sv.SV_ERR_NULL, name
    for kw in (dict(n_rows=-1), dict(n_req=-1), dict(max_pages=-1), dict(latent_ld=504),
               dict(latent_ld=516), dict(rope_ld=56), dict(rope_ld=68), dict(latent=ODD),
               dict(rope=ODD), dict(n_rows=sv.SV_MAX_APPEND_VALUES // 576 + 1),
               dict(max_pages=sv.SV_MAX_CONTEXT // 16 + 1), dict(latent_ld=2 ** 60)):
        assert append(**kw) == sv.SV_ERR_SHAPE, kw
    for name in ("table", "q", "cu", "ctx", "out"):
        assert attend(**{name: None}) == sv.SV_ERR_NULL, name
    for kw in (dict(n_req=-1), dict(k_max=-1), dict(k_max=sv.SV_MAX_DRAFT + 1), dict(n_heads=0),
               dict(q_ld=16 * 576 - 8), dict(q_ld=16 * 576 + 4), dict(out_ld=16 * 512 - 8),
               dict(q=ODD), dict(out=ODD), dict(q_rows=-1), dict(q_rows=2 ** 31), dict(max_pages=-1),
               dict(n_req=sv.SV_MAX_ATTEND_SLOTS), dict(q_ld=2 ** 60),
               dict(max_pages=sv.SV_MAX_CONTEXT // 16 + 1)):
        assert attend(**kw) == sv.SV_ERR_SHAPE, kw
    assert attend(latent(n_pages=0)) == sv.SV_ERR_SHAPE
    for scale in (math.inf, -math.inf, math.nan):
        assert attend(scale=scale) == sv.SV_ERR_VALUE
    # nothing to do needs nothing
    assert append(n_rows=0, latent=None) == attend(n_req=0, q=None) == sv.SV_OK


def test_latent_workspaces():
    f = sv.sv_latent_attend_workspace_bytes
    need = f(2, 3, 16, 512, 1000, 16)
    assert need > 0 and need % 4 == 0
    for kw in (dict(ws=None, ws_bytes=need), dict(ws_bytes=need - 1),
               dict(ws=ODD, ws_bytes=need)):
        assert attend(max_pages=1000, **kw) == sv.SV_ERR_WORKSPACE, kw
    assert f(512, 3, 128, 512, 1000, 16) == 0  # one part each
    for bad in ((-1, 3, 16, 512, 4, 16), (2, 65, 16, 512, 4, 16), (2, 3, 0, 512, 4, 16),
                (2, 3, 16, 128, 4, 16), (2, 3, 16, 512, -1, 16), (2, 3, 16, 512, 4, 0),
                (2, 3, 16, 512, 2 ** 31 - 1, 2 ** 31 - 1)):
        assert f(*bad) == 0


@pytest.mark.parametrize("kw", [dict(head_dim=96), dict(n_kv_heads=0), dict(n_pages=-1),
                                dict(page_size=0), dict(page_stride=4), dict(token_stride=-8),
                                dict(k=0x1008), dict(v=0x1008), dict(n_pages=0)])
def test_shared_layouts(kw):
    assert shared(cache(**kw)) == sv.SV_ERR_SHAPE


def test_shared_refusals():
    assert shared(ctypes.c_void_p(None)) == sv.SV_ERR_NULL
    assert shared(cache(dtype=sv.SV_F32)) == sv.SV_ERR_DTYPE
    assert shared(cache(k=None)) == shared(cache(v=None)) == sv.SV_ERR_NULL
    for name in ("table", "q", "cu", "ctx", "out", "start", "prefix"):
        assert shared(**{name: None}) == sv.SV_ERR_NULL, name
    for kw in (dict(n_groups=-1), dict(n_groups=3), dict(n_req=-1), dict(k_max=-1),
               dict(k_max=sv.SV_MAX_DRAFT + 1), dict(n_heads=1), dict(n_heads=5), dict(q_ld=248),
               dict(q_ld=260), dict(out_ld=248), dict(q=ODD), dict(out=ODD), dict(q_rows=-1),
               dict(q_rows=2 ** 31), dict(max_pages=-1), dict(n_req=sv.SV_MAX_ATTEND_SLOTS),
               dict(q_ld=2 ** 60), dict(max_pages=sv.SV_MAX_CONTEXT // 16 + 1)):
        assert shared(**kw) == sv.SV_ERR_SHAPE, kw
    for scale in (math.inf, math.nan):
        assert shared(scale=scale) == sv.SV_ERR_VALUE
    # without groups their arrays are not asked for: the workspace is the next refusal
    assert shared(n_groups=0, start=None, prefix=None) == sv.SV_ERR_WORKSPACE
    assert shared(n_req=0, n_groups=0, q=None) == sv.SV_OK


def test_shared_workspaces():
    f = sv.sv_cache_attend_shared_workspace_bytes
    need = f(2, 1, 3, 4, 2, 64, 4, 16)
    assert need > 0
    for kw in (dict(ws=None, ws_bytes=need), dict(ws_bytes=need - 1), dict(ws=ODD, ws_bytes=need)):
        assert shared(**kw) == sv.SV_ERR_WORKSPACE, kw
    for bad in ((2, 3, 3, 4, 2, 64, 4, 16), (2, -1, 3, 4, 2, 64, 4, 16), (2, 1, 65, 4, 2, 64, 4, 16),
                (2, 1, 3, 5, 2, 64, 4, 16), (2, 1, 3, 4, 2, 96, 4, 16), (2, 1, 3, 4, 2, 64, -1, 16),
                (2, 1, 3, 4, 2, 64, 4, 0)):
        assert f(*bad) == 0, bad


def test_the_binding_refuses():
    with pytest.raises((TypeError, ValueError)):  # not on a GPU
        sv.LatentCache(torch.zeros(2, 4, 576, dtype=torch.bfloat16), 512)
    with pytest.raises((TypeError, ValueError)):
        sv.PagedCache(torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16),
                      torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16))


def test_the_latent_oracle_against_plain_attention():
    """The absorbed form is attention with one kv head whose keys are the vectors and whose
    values their first dims; what was appended is what is read."""
    g = np.random.default_rng(5)
    rank, dim, heads, size = 256, 320, 3, 4
    table = np.array([[2, 0, 5], [4, 1, 3]])
    ctx, cu = np.array([5, 2]), np.array([0, 2, 5])
    kv = np.asarray(g.standard_normal((6, size, dim)), np.float32)
    rows = np.asarray(g.standard_normal((5, dim)), np.float32)
    req, pos = [0, 0, 1, 1, 1], [0, 1, 0, 1, 2]
    kv = latent_append(kv, table, rows[:, :rank], rows[:, rank:], req, pos, ctx)
    for i in range(5):
        t = ctx[req[i]] + pos[i]
        np.testing.assert_array_equal(kv[table[req[i], t // size], t % size], rows[i])
    q = g.standard_normal((5, heads, dim))
    out, lse, _ = latent_attend(q, kv, rank, table, cu, ctx, 0.2)
    want, want_lse, _ = cache_attend(q, kv[:, :, None], kv[:, :, None], table, cu, ctx, 0.2)
    np.testing.assert_allclose(out, want[..., :rank], rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(lse, want_lse, rtol=1e-12)


def test_host_sides_under_sanitizers(tmp_path):
    """The API files built with g++ under ASan and UBSan against stub launchers."""
    gxx = shutil.which("g++")
    driver = os.path.join(HERE, "latent_asan_driver.cpp")
    if gxx is None or not os.path.exists(driver) or \
            not os.path.exists(os.path.join(ROCM, "include", "hip", "hip_runtime.h")):
        pytest.skip("g++, the driver or the HIP headers are not available")
    exe = tmp_path / "latent_checks"
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer",
           "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined",
           "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           "-I", os.path.join(ROCM, "include"),
           *[os.path.join(CSRC, f"sv_{n}_api.cpp") for n in ("logits", "latent", "shared")], driver,
           "-o", str(exe)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0")
    run = subprocess.run([str(exe)], capture_output=True, text=True, env=env, timeout=120)
    assert run.returncode == 0, run.stdout[-2000:] + run.stderr[-4000:]
    assert "latent and shared checks passed" in run.stdout
