"""Host validation of the sampling, truncated verification and paged cache
calls (CPU): refusals come before anything is launched, passing arguments reach
the launch checks, and the binding refuses what does not fit."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

sv = pytest.importorskip("adaptive_draft_verification_amd",
                         reason="libspecverify.so not built (python adaptive_draft_verification_amd/build.py)")

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "adaptive_draft_verification_amd", "csrc")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p(0x1001)


def sample(**kw):
    args = dict(logits=FAKE, ld=64, n_rows=4, dtype=sv.SV_BF16, vocab=64, law=None, u=FAKE,
                tokens=FAKE, prob=None, support=None, dev_error=None, stream=None)
    args.update(kw)
    return sv._lib.sv_sample(*args.values())


def test_sample_refusals():
    assert sample(dtype=sv.SV_E4M3) == sv.SV_ERR_DTYPE
    assert sample(dtype=9) == sv.SV_ERR_DTYPE
    for kw in (dict(n_rows=-1), dict(n_rows=sv.SV_MAX_SAMPLE_ROWS + 1), dict(vocab=0),
               dict(vocab=sv.SV_MAX_VOCAB + 1, ld=2 ** 21), dict(ld=63), dict(ld=2 ** 60),
               dict(logits=ODD), dict(logits=ctypes.c_void_p(0x1002), dtype=sv.SV_F32)):
        assert sample(**kw) == sv.SV_ERR_SHAPE, kw
    for key in ("logits", "u", "tokens"):
        assert sample(**{key: None}) == sv.SV_ERR_NULL, key
    assert sample(n_rows=0, logits=None, u=None, tokens=None) == sv.SV_OK
    assert sv.SV_MAX_SAMPLE_ROWS * 1024 < 2 ** 32


def verify(**kw):
    args = dict(target=FAKE, target_ld=64, target_rows=16, draft=FAKE, draft_ld=64,
                dtype=sv.SV_F32, vocab=64, draft_tokens=FAKE, cu_rows=FAKE, n_req=4, k_max=3,
                target_law=None, draft_law=None, seed=0, step=0, tokens=FAKE, accepted=FAKE,
                p=None, q=None, mass=None, dev_error=None, ws=FAKE,
                ws_bytes=sv.sv_verify_truncated_workspace_bytes(4, 3), stream=None)
    args.update(kw)
    return sv._lib.sv_verify_truncated(*args.values())


def test_verify_truncated_refusals():
    assert sv.sv_verify_truncated_workspace_bytes(4, 3) == 4 * (7 * 32 + 8 * 8)
    for n, k in ((-1, 3), (1, 65), (1, -1), (sv.SV_MAX_VERIFY_SLOTS // 15 + 1, 7)):
        assert sv.sv_verify_truncated_workspace_bytes(n, k) == 0
        assert verify(n_req=n, k_max=k) == sv.SV_ERR_SHAPE
    assert verify(dtype=sv.SV_E4M3) == sv.SV_ERR_DTYPE
    for kw in (dict(vocab=0), dict(target_ld=63), dict(draft_ld=63), dict(target_rows=-1),
               dict(vocab=sv.SV_MAX_VOCAB + 1, target_ld=2 ** 21, draft_ld=2 ** 21),
               dict(target=ODD), dict(draft=ctypes.c_void_p(0x1002)),
               dict(target_ld=2 ** 60), dict(draft_ld=2 ** 60)):
        assert verify(**kw) == sv.SV_ERR_SHAPE, kw
    for key in ("target", "cu_rows", "tokens", "accepted", "draft_tokens", "draft"):
        assert verify(**{key: None}) == sv.SV_ERR_NULL, key
    need = sv.sv_verify_truncated_workspace_bytes(4, 3)
    for kw in (dict(ws=None), dict(ws_bytes=need - 1), dict(ws=ctypes.c_void_p(0x1004))):
        assert verify(**kw) == sv.SV_ERR_WORKSPACE, kw
    # no drafts: their rows and ids are not needed
    assert verify(k_max=0, draft=None, draft_ld=0, draft_tokens=None, ws=None) == \
        sv.SV_ERR_WORKSPACE
    assert verify(n_req=0, target=None, ws=None) == sv.SV_OK


def cache(**kw):
    args = dict(k=0x1000, v=0x2000, dtype=sv.SV_BF16, n_pages=8, page_size=16, n_kv_heads=2,
                head_dim=64, page_stride=16 * 128, token_stride=128, head_stride=64,
                k_scale=None, v_scale=None)
    args.update(kw)
    return ctypes.byref(sv._Cache(*args.values()))


BAD_CACHES = [(dict(dtype=sv.SV_F32), "SV_ERR_DTYPE"), (dict(dtype=7), "SV_ERR_DTYPE")] + [
    (kw, "SV_ERR_SHAPE") for kw in (
        dict(head_dim=96), dict(head_dim=0), dict(n_pages=-1), dict(page_size=0),
        dict(n_kv_heads=0), dict(page_stride=4), dict(token_stride=-128), dict(head_stride=65),
        dict(dtype=sv.SV_E4M3, head_stride=8), dict(k=0x1008), dict(v=0x1002),
        dict(page_stride=2 ** 60), dict(page_size=2 ** 30))]


def append(c=None, **kw):
    args = dict(table=FAKE, max_pages=4, k=FAKE, v=FAKE, kv_ld=128, row_req=FAKE, row_pos=FAKE,
                n_rows=8, ctx_len=FAKE, n_req=2, dev_error=None, stream=None)
    args.update(kw)
    return sv._lib.sv_cache_append(cache() if c is None else c, *args.values())


def attend(c=None, **kw):
    args = dict(table=FAKE, max_pages=4, q=FAKE, q_ld=256, q_rows=8, n_heads=4, cu_rows=FAKE,
                ctx_len=FAKE, n_req=2, k_max=3, scale=0.125, out=FAKE, out_ld=256, lse=None,
                dev_error=None, ws=None, ws_bytes=0, stream=None)
    args.update(kw)
    return sv._lib.sv_cache_attend(cache() if c is None else c, *args.values())


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_cache_layout_refusals(kw, status):
    assert append(cache(**kw)) == getattr(sv, status)
    assert attend(cache(**kw)) == getattr(sv, status)


def test_cache_append_refusals():
    assert append(ctypes.c_void_p(None)) == sv.SV_ERR_NULL
    assert attend(ctypes.c_void_p(None)) == sv.SV_ERR_NULL
    for kw in (dict(max_pages=-1), dict(n_rows=-1), dict(n_req=-1), dict(kv_ld=127),
               dict(kv_ld=132), dict(kv_ld=2 ** 60), dict(k=ODD), dict(v=ODD),
               dict(n_rows=2 ** 30)):
        assert append(**kw) == sv.SV_ERR_SHAPE, kw
    for key in ("table", "k", "v", "row_req", "row_pos", "ctx_len"):
        assert append(**{key: None}) == sv.SV_ERR_NULL, key
    assert append(cache(k=None)) == sv.SV_ERR_NULL
    assert append(n_rows=0, k=None, v=None) == sv.SV_OK
    assert append(n_req=0, k=None, v=None) == sv.SV_OK


def test_cache_attend_refusals():
    for kw in (dict(max_pages=-1), dict(n_req=-1), dict(k_max=-1), dict(k_max=65),
               dict(n_heads=3), dict(n_heads=0), dict(q_rows=-1), dict(q_rows=2 ** 31),
               dict(q_ld=255), dict(q_ld=260), dict(out_ld=2 ** 60), dict(q=ODD), dict(out=ODD),
               dict(n_req=2 ** 22)):
        assert attend(**kw) == sv.SV_ERR_SHAPE, kw
    assert attend(cache(n_pages=0)) == sv.SV_ERR_SHAPE
    for scale in (float("nan"), float("inf")):
        assert attend(scale=scale) == sv.SV_ERR_VALUE
    for key in ("table", "q", "cu_rows", "ctx_len", "out"):
        assert attend(**{key: None}) == sv.SV_ERR_NULL, key
    assert attend(n_req=0, q=None, out=None) == sv.SV_OK
    need = sv.sv_cache_attend_workspace_bytes(2, 3, 4, 2, 64, 1024, 16)
    assert need > 0 and need % 4 == 0
    for kw in (dict(ws=None), dict(ws=FAKE, ws_bytes=need - 1),
               dict(ws=ctypes.c_void_p(0x1008), ws_bytes=need)):
        assert attend(max_pages=1024, **kw) == sv.SV_ERR_WORKSPACE, kw
    assert sv.SV_MAX_ATTEND_SLOTS * 256 <= 2 ** 32


def test_cache_attend_workspace_sizes():
    f = sv.sv_cache_attend_workspace_bytes
    # one workgroup's worth of positions, or enough requests: the length is not split
    assert f(1, 0, 8, 8, 128, 4, 16) == 0
    assert f(1024, 0, 8, 8, 128, 1000, 16) == 0
    # else head_dim + 2 floats for each row, head and part
    b = f(1, 0, 8, 8, 128, 10000, 16)
    assert b > 0 and b % (8 * 130 * 4) == 0 and b // (8 * 130 * 4) <= 128
    for bad in ((-1, 0, 8, 8, 128, 4, 16), (1, 65, 8, 8, 128, 4, 16), (1, 0, 7, 2, 128, 4, 16),
                (1, 0, 8, 8, 100, 4, 16), (1, 0, 8, 8, 128, -1, 16), (1, 0, 8, 8, 128, 4, 0)):
        assert f(*bad) == 0, bad


def test_binding_refuses_host_tensors():
    z = torch.zeros(2, 8)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        sv.sv_sample(z, torch.zeros(2), None, i)
    with pytest.raises(ValueError):
        sv.PagedCache(torch.zeros(1, 16, 1, 64, dtype=torch.bfloat16),
                      torch.zeros(1, 16, 1, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        sv.sv_verify_truncated(z, z, i[:, None], i, None, None, 0, 0, i[:, None], i, None)


def test_serving_host_side_under_sanitizers(tmp_path):
    """The two API files built with g++ under ASan and UBSan against stub launchers."""
    gxx = shutil.which("g++")
    driver = os.path.join(HERE, "serve_asan_driver.cpp")
    if gxx is None or not os.path.exists(driver) or \
            not os.path.exists(os.path.join(ROCM, "include", "hip", "hip_runtime.h")):
        pytest.skip("g++, the driver or the HIP headers are not available")
    exe = tmp_path / "serve_checks"
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer",
           "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined",
           "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           "-I", os.path.join(ROCM, "include"), os.path.join(CSRC, "sv_sample_api.cpp"),
           os.path.join(CSRC, "sv_cache_api.cpp"), driver, "-o", str(exe)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0")
    run = subprocess.run([str(exe)], capture_output=True, text=True, env=env, timeout=120)
    assert run.returncode == 0, run.stdout[-2000:] + run.stderr[-4000:]
    assert "serving checks passed" in run.stdout


def test_cache_sizes_at_the_limits():
    f = sv.sv_cache_attend_workspace_bytes
    heads = sv.SV_MAX_ATTEND_SLOTS + 1
    assert heads * 256 == 2 ** 32   # one workgroup a slot would pass a grid's limit
    for kw in (dict(n_req=heads, k_max=0, n_heads=2), dict(n_req=heads // 4, k_max=0),
               dict(n_req=1, k_max=0, n_heads=heads, q_ld=64 * heads, out_ld=64 * heads)):
        assert attend(**kw) == sv.SV_ERR_SHAPE, kw
    # no request, but sizes whose product passes 32 bits
    assert f(0, 64, 2 ** 31 - 1, 1, 64, 4, 16) == 0
    assert attend(cache(n_kv_heads=1), n_req=0, k_max=64, n_heads=2 ** 31 - 1) == sv.SV_ERR_SHAPE
    # positions and a tile past the last one count in 32 bits
    assert sv.SV_MAX_CONTEXT + 65536 == 2 ** 31
    pages = sv.SV_MAX_CONTEXT // 16
    assert f(1, 0, 1, 1, 64, pages, 16) > 0
    assert f(1, 0, 1, 1, 64, pages + 1, 16) == 0
    assert attend(max_pages=pages) == sv.SV_ERR_WORKSPACE
    assert attend(max_pages=pages + 1) == sv.SV_ERR_SHAPE
    assert append(max_pages=pages + 1) == sv.SV_ERR_SHAPE
