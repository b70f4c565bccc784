"""Python binding of libspecverify (argument marshalling only).

Every step of the verify path runs in the HIP kernels of libspecverify.so,
built in-tree by ``adaptive_draft_verification_amd/build.py``.  PyTorch supplies
device memory and streams; nothing here computes.  Importing this module
fails loudly if the library has not been built: there is no fallback.

The functions keep the C names (sv_budget_select, sv_pack_varlen, sv_verify,
...) and take torch tensors; shapes are read from the tensors, the stream is
torch's current stream unless one is given.  A non-OK status raises SvError.
"""

import ctypes
import os
from typing import NamedTuple, Optional

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspecverify.so")

SV_OK, SV_ERR_NULL, SV_ERR_SHAPE, SV_ERR_DTYPE, SV_ERR_VALUE, SV_ERR_WORKSPACE, SV_ERR_LAUNCH, \
    SV_ERR_CAPACITY, SV_ERR_DATA = range(9)
SV_F32, SV_BF16, SV_E4M3 = 0, 1, 2
SV_STOCHASTIC, SV_GREEDY = 0, 1
SV_DEV_BAD_CU_ROWS, SV_DEV_BAD_TOKEN, SV_DEV_NONFINITE = 1, 2, 4
SV_DEV_BAD_DRAFT_LEN, SV_DEV_BAD_COST, SV_DEV_BAD_KEPT = 8, 16, 32
SV_DEV_BAD_PAGE, SV_DEV_BAD_CTX, SV_DEV_BAD_PARAM, SV_DEV_BAD_SLOT = 64, 128, 256, 512
SV_MAX_BUDGET_SLOTS, SV_MAX_DRAFT, SV_MAX_VOCAB = 8192, 64, 1048576
SV_MAX_VERIFY_SLOTS = 524288
SV_NOALLOC_WS_BYTES = 8388608
SV_MAX_ATTEND_SLOTS, SV_MAX_CONTEXT = 16777215, 2147418112
SV_MAX_APPEND_VALUES = 1073741824
SV_MAX_SAMPLE_ROWS = 4194303
SV_LATENT_ROPE = 64
SV_MAX_HISTORY_TOKENS, SV_MAX_ADJUST_PARTS = 1073741824, 16777215

EXPORTED = ["sv_status_str", "sv_budget_workspace_bytes", "sv_verify_workspace_bytes",
            "sv_cost_table_prepare", "sv_budget_select", "sv_budget_allocate",
            "sv_budget_select_pack", "sv_budget_allocate_pack",
            "sv_uniform_k_select", "sv_pack_varlen",
            "sv_verify",
            "sv_verify_stages", "sv_verify_noalloc", "sv_accept_stats", "sv_calibrate_update", "sv_calibrate_predict",
            "sv_philox_uniforms",
            "sv_cache_append", "sv_cache_attend", "sv_cache_attend_workspace_bytes",
            "sv_sample", "sv_verify_truncated", "sv_verify_truncated_workspace_bytes",
            "sv_history_clear", "sv_history_add", "sv_adjust_logits",
            "sv_latent_append", "sv_latent_attend", "sv_latent_attend_workspace_bytes",
            "sv_cache_attend_shared", "sv_cache_attend_shared_workspace_bytes"]


class _Cache(ctypes.Structure):
    """sv_cache of the C header."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int),
                ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p)]


class _Law(ctypes.Structure):
    """sv_sampling of the C header."""
    _fields_ = [("temperature", ctypes.c_void_p), ("top_k", ctypes.c_void_p),
                ("top_p", ctypes.c_void_p), ("min_p", ctypes.c_void_p)]


class _LatentCache(ctypes.Structure):
    """sv_latent_cache of the C header."""
    _fields_ = [("kv", ctypes.c_void_p), ("dtype", ctypes.c_int), ("n_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("latent_dim", ctypes.c_int32),
                ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("scale", ctypes.c_void_p)]


class _History(ctypes.Structure):
    """sv_history of the C header."""
    _fields_ = [("counts", ctypes.c_void_p), ("seen", ctypes.c_void_p),
                ("n_seen", ctypes.c_void_p), ("n_slots", ctypes.c_int32),
                ("vocab", ctypes.c_int32), ("cap", ctypes.c_int32)]


class _Penalties(ctypes.Structure):
    """sv_penalties of the C header."""
    _fields_ = [("repetition", ctypes.c_void_p), ("frequency", ctypes.c_void_p),
                ("presence", ctypes.c_void_p)]


class _Bias(ctypes.Structure):
    """sv_bias of the C header."""
    _fields_ = [("start", ctypes.c_void_p), ("ids", ctypes.c_void_p),
                ("values", ctypes.c_void_p), ("n_entries", ctypes.c_int32)]


class _TokenMask(ctypes.Structure):
    """sv_token_mask of the C header."""
    _fields_ = [("bits", ctypes.c_void_p), ("ld", ctypes.c_int64), ("n_masks", ctypes.c_int32),
                ("row_mask", ctypes.c_void_p)]


class SvError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {_lib.sv_status_str(status).decode()} (status {status})")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python adaptive_draft_verification_amd/build.py` "
                          "(there is no non-HIP fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, u64, f32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                                  ctypes.c_uint64, ctypes.c_float, ctypes.c_size_t)
    sig = {
        "sv_status_str": (ctypes.c_char_p, [ctypes.c_int]),
        "sv_budget_workspace_bytes": (sz, [i32, i32]),
        "sv_verify_workspace_bytes": (sz, [i32, i32]),
        "sv_cost_table_prepare": (ctypes.c_int, [vp, i32, i32, vp, i32]),
        "sv_budget_select": (ctypes.c_int, [vp, vp, i32, i32, vp, i32, i32, i32, vp, vp, vp, vp,
                                            vp, sz, vp]),
        "sv_budget_allocate": (ctypes.c_int, [vp, vp, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp]),
        "sv_budget_select_pack": (ctypes.c_int, [vp, vp, i32, i32, vp, i32, i32, i32, vp, vp, vp,
                                                 vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "sv_budget_allocate_pack": (ctypes.c_int, [vp, vp, i32, i32, vp, vp, vp, vp, vp, vp, vp,
                                                   vp, vp, vp, vp, vp, sz, vp]),
        "sv_uniform_k_select": (ctypes.c_int, [vp, vp, i32, i32, vp, i32, i32, i32, vp, vp, vp,
                                               vp, vp]),
        "sv_pack_varlen": (ctypes.c_int, [vp, vp, vp, i32, i32, vp, vp, vp, vp, vp, vp]),
        "sv_verify": (ctypes.c_int, [vp, i64, i64, vp, i64, ctypes.c_int, i32, vp, vp, i32, i32,
                                     ctypes.c_int, f32, u64, u64, vp, vp, vp, vp, vp, vp, vp, vp,
                                     vp, sz, vp]),
        "sv_verify_stages": (ctypes.c_int, [vp, i64, i64, vp, i64, ctypes.c_int, i32, vp, vp, i32,
                                            i32, ctypes.c_int, f32, u64, u64, vp, vp, vp, vp, vp,
                                            vp, vp, vp, vp, sz, i32, vp]),
        "sv_verify_noalloc": (ctypes.c_int, [vp, i64, i64, vp, i64, ctypes.c_int, i32, vp, vp,
                                             i32, i32, ctypes.c_int, f32, u64, u64, vp, vp, vp,
                                             vp, vp, vp, vp, vp, vp]),
        "sv_accept_stats": (ctypes.c_int, [vp, vp, i32, i32, vp, vp, vp, vp]),
        "sv_calibrate_update": (ctypes.c_int, [vp, vp, vp, vp, vp, vp, i32, i32, f32, vp, vp]),
        "sv_calibrate_predict": (ctypes.c_int, [vp, vp, vp, vp, i32, i32, vp, vp]),
        "sv_philox_uniforms": (ctypes.c_int, [u64, u64, i32, i32, vp, vp, vp]),
        "sv_cache_append": (ctypes.c_int, [vp, vp, i32, vp, vp, i64, vp, vp, i32, vp, i32, vp,
                                           vp]),
        "sv_cache_attend_workspace_bytes": (sz, [i32, i32, i32, i32, i32, i32, i32]),
        "sv_cache_attend": (ctypes.c_int, [vp, vp, i32, vp, i64, i64, i32, vp, vp, i32, i32, f32,
                                           vp, i64, vp, vp, vp, sz, vp]),
        "sv_sample": (ctypes.c_int, [vp, i64, i32, ctypes.c_int, i32, vp, vp, vp, vp, vp, vp, vp]),
        "sv_verify_truncated_workspace_bytes": (sz, [i32, i32]),
        "sv_verify_truncated": (ctypes.c_int, [vp, i64, i64, vp, i64, ctypes.c_int, i32, vp, vp,
                                               i32, i32, vp, vp, u64, u64, vp, vp, vp, vp, vp, vp,
                                               vp, sz, vp]),
        "sv_cache_attend_shared_workspace_bytes": (sz, [i32, i32, i32, i32, i32, i32, i32, i32]),
        "sv_cache_attend_shared": (ctypes.c_int, [vp, vp, i32, vp, i64, i64, i32, vp, vp, i32, i32,
                                                  vp, vp, i32, f32, vp, i64, vp, vp, vp, sz, vp]),
        "sv_latent_append": (ctypes.c_int, [vp, vp, i32, vp, i64, vp, i64, vp, vp, i32, vp, i32, vp,
                                            vp]),
        "sv_latent_attend_workspace_bytes": (sz, [i32, i32, i32, i32, i32, i32]),
        "sv_latent_attend": (ctypes.c_int, [vp, vp, i32, vp, i64, i64, i32, vp, vp, i32, i32, f32,
                                            vp, i64, vp, vp, vp, sz, vp]),
        "sv_history_clear": (ctypes.c_int, [vp, vp, i32, vp, vp]),
        "sv_history_add": (ctypes.c_int, [vp, vp, vp, i64, i32, i32, i32, vp, vp]),
        "sv_adjust_logits": (ctypes.c_int, [vp, i64, vp, i64, i32, ctypes.c_int, i32, vp, vp, i32,
                                            i32, vp, vp, vp, vp, vp, vp, vp, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


# The serving calls below run every decode step, some of them many times: their
# checks are written for few Python operations (addresses go to the library as
# plain integers, devices are compared by index).

def _on(t, dtype, name, device, shape):
    """Address of a contiguous device tensor of this type, device and shape (None: no tensor)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
        _dev(t, dtype, name)
        raise ValueError(f"{name} must be on the call's device")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _launch(fn, name, device, stream, *args):
    """fn(*args, stream) with `device` current; stream: the given one, else the device's current."""
    if stream is None:
        handle = (_raw_stream(device) if _raw_stream is not None
                  else torch.cuda.current_stream(device).cuda_stream)
    elif stream.device.index != device:
        raise ValueError("the stream must be on the tensors' device")
    else:
        handle = stream.cuda_stream
    current = torch.cuda.current_device()
    if current == device:
        status = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            status = fn(*args, handle)
    if status != SV_OK:
        raise SvError(status, name)


def _dev(t, dtype, name, ndim=None):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")


def _check(status, where):
    if status != SV_OK:
        raise SvError(status, where)


def sv_status_str(status):
    return _lib.sv_status_str(status).decode()


def sv_budget_workspace_bytes(n_req, k_max):
    return int(_lib.sv_budget_workspace_bytes(n_req, k_max))


def sv_verify_workspace_bytes(n_req, k_max):
    return int(_lib.sv_verify_workspace_bytes(n_req, k_max))


def sv_cost_table_prepare(raw, granule, out_len):
    """Host call: shaped cost table (numpy fp32 in, numpy fp32 out)."""
    raw = np.ascontiguousarray(raw, dtype=np.float32)
    out = np.zeros(int(out_len), dtype=np.float32)
    _check(_lib.sv_cost_table_prepare(raw.ctypes.data_as(ctypes.c_void_p), len(raw), int(granule),
                                      out.ctypes.data_as(ctypes.c_void_p), int(out_len)),
           "sv_cost_table_prepare")
    return out


def sv_budget_select(conf, draft_len, cost, t_base, n_bonus, kept, budget, survival=None,
                     dev_error=None, stream=None, ws=None):
    """conf [n, k_max] f32, draft_len [n] i32, cost [L] f32 -> kept [n] i32, budget [1] i32.

    ws: device uint8 tensor of at least sv_budget_workspace_bytes(n, k_max) bytes."""
    _dev(conf, torch.float32, "conf", 2)
    _dev(draft_len, torch.int32, "draft_len", 1)
    _dev(cost, torch.float32, "cost", 1)
    _dev(kept, torch.int32, "kept", 1)
    _dev(budget, torch.int32, "budget", 1)
    _dev(survival, torch.float32, "survival", 2)
    _dev(dev_error, torch.int32, "dev_error", 1)
    _dev(ws, torch.uint8, "ws", 1)
    n, k_max = conf.shape
    if draft_len.numel() != n or kept.numel() != n or budget.numel() < 1:
        raise ValueError("draft_len, kept must have n entries and budget one")
    if survival is not None and tuple(survival.shape) != (n, k_max):
        raise ValueError("survival must be [n, k_max]")
    _check(_lib.sv_budget_select(_ptr(conf), _ptr(draft_len), n, k_max, _ptr(cost), cost.numel(),
                                 int(t_base), int(n_bonus), _ptr(kept), _ptr(budget),
                                 _ptr(survival), _ptr(dev_error), _ptr(ws), 0 if ws is None else ws.numel(),
                                 _stream(stream)),
           "sv_budget_select")


def sv_budget_allocate(conf, draft_len, budget_in, kept, budget_used=None, survival=None,
                       dev_error=None, stream=None, ws=None):
    """conf [n, k_max] f32, draft_len [n] i32, budget_in [1] i32 (device) -> kept [n] i32.

    ws: device uint8 tensor of at least sv_budget_workspace_bytes(n, k_max) bytes."""
    _dev(conf, torch.float32, "conf", 2)
    _dev(draft_len, torch.int32, "draft_len", 1)
    _dev(budget_in, torch.int32, "budget_in", 1)
    _dev(kept, torch.int32, "kept", 1)
    _dev(budget_used, torch.int32, "budget_used", 1)
    _dev(survival, torch.float32, "survival", 2)
    _dev(dev_error, torch.int32, "dev_error", 1)
    _dev(ws, torch.uint8, "ws", 1)
    n, k_max = conf.shape
    if draft_len.numel() != n or kept.numel() != n or budget_in.numel() < 1:
        raise ValueError("draft_len, kept must have n entries and budget_in one")
    if survival is not None and tuple(survival.shape) != (n, k_max):
        raise ValueError("survival must be [n, k_max]")
    _check(_lib.sv_budget_allocate(_ptr(conf), _ptr(draft_len), n, k_max, _ptr(budget_in),
                                   _ptr(kept), _ptr(budget_used), _ptr(survival), _ptr(dev_error),
                                   _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)),
           "sv_budget_allocate")


def _pack_outputs(n, k_max, last_token, draft_tokens, cu_rows, row_req, row_pos, packed_tokens):
    for name, t in (("last_token", last_token), ("cu_rows", cu_rows), ("row_req", row_req),
                    ("row_pos", row_pos), ("packed_tokens", packed_tokens)):
        _dev(t, torch.int32, name, 1)
    _dev(draft_tokens, torch.int32, "draft_tokens", 2)
    cap = n * (k_max + 1)
    if tuple(draft_tokens.shape) != (n, k_max) or last_token.numel() != n \
            or cu_rows.numel() != n + 1:
        raise ValueError("draft_tokens [n, k_max], last_token [n], cu_rows [n+1]")
    if row_req.numel() != cap or row_pos.numel() != cap or packed_tokens.numel() != cap:
        raise ValueError("row maps need n*(k_max+1) entries")


def sv_budget_select_pack(conf, draft_len, cost, t_base, n_bonus, last_token, draft_tokens, kept,
                          budget, cu_rows, row_req, row_pos, packed_tokens, survival=None,
                          dev_error=None, stream=None, ws=None):
    """sv_budget_select then sv_pack_varlen, one launch fewer (same tensors as the two)."""
    for name, t, nd in (("conf", conf, 2), ("draft_len", draft_len, 1), ("cost", cost, 1),
                        ("kept", kept, 1), ("budget", budget, 1)):
        _dev(t, torch.float32 if name in ("conf", "cost") else torch.int32, name, nd)
    _dev(survival, torch.float32, "survival", 2)
    _dev(dev_error, torch.int32, "dev_error", 1)
    _dev(ws, torch.uint8, "ws", 1)
    n, k_max = conf.shape
    if draft_len.numel() != n or kept.numel() != n or budget.numel() < 1:
        raise ValueError("draft_len, kept must have n entries and budget one")
    _pack_outputs(n, k_max, last_token, draft_tokens, cu_rows, row_req, row_pos, packed_tokens)
    _check(_lib.sv_budget_select_pack(_ptr(conf), _ptr(draft_len), n, k_max, _ptr(cost),
                                      cost.numel(), int(t_base), int(n_bonus), _ptr(last_token),
                                      _ptr(draft_tokens), _ptr(kept), _ptr(budget),
                                      _ptr(survival), _ptr(cu_rows), _ptr(row_req), _ptr(row_pos),
                                      _ptr(packed_tokens), _ptr(dev_error), _ptr(ws),
                                      0 if ws is None else ws.numel(), _stream(stream)),
           "sv_budget_select_pack")


def sv_budget_allocate_pack(conf, draft_len, budget_in, last_token, draft_tokens, kept, cu_rows,
                            row_req, row_pos, packed_tokens, budget_used=None, survival=None,
                            dev_error=None, stream=None, ws=None):
    """sv_budget_allocate then sv_pack_varlen, one launch fewer."""
    _dev(conf, torch.float32, "conf", 2)
    for name, t in (("draft_len", draft_len), ("budget_in", budget_in), ("kept", kept),
                    ("budget_used", budget_used), ("dev_error", dev_error)):
        _dev(t, torch.int32, name, 1)
    _dev(survival, torch.float32, "survival", 2)
    _dev(ws, torch.uint8, "ws", 1)
    n, k_max = conf.shape
    if draft_len.numel() != n or kept.numel() != n or budget_in.numel() < 1:
        raise ValueError("draft_len, kept must have n entries and budget_in one")
    _pack_outputs(n, k_max, last_token, draft_tokens, cu_rows, row_req, row_pos, packed_tokens)
    _check(_lib.sv_budget_allocate_pack(_ptr(conf), _ptr(draft_len), n, k_max, _ptr(budget_in),
                                        _ptr(last_token), _ptr(draft_tokens), _ptr(kept),
                                        _ptr(budget_used), _ptr(survival), _ptr(cu_rows),
                                        _ptr(row_req), _ptr(row_pos), _ptr(packed_tokens),
                                        _ptr(dev_error), _ptr(ws),
                                        0 if ws is None else ws.numel(), _stream(stream)),
           "sv_budget_allocate_pack")


def sv_uniform_k_select(conf, draft_len, cost, t_base, n_bonus, kept, k_out, scores=None,
                        dev_error=None, stream=None):
    """conf [n, k_max] f32, draft_len [n] i32, cost [L] f32 -> kept [n] i32, k_out [1] i32,
    scores [k_max + 1] f64 (optional)."""
    _dev(conf, torch.float32, "conf", 2)
    _dev(draft_len, torch.int32, "draft_len", 1)
    _dev(cost, torch.float32, "cost", 1)
    _dev(kept, torch.int32, "kept", 1)
    _dev(k_out, torch.int32, "k_out", 1)
    _dev(scores, torch.float64, "scores", 1)
    _dev(dev_error, torch.int32, "dev_error", 1)
    n, k_max = conf.shape
    if draft_len.numel() != n or kept.numel() != n or k_out.numel() < 1:
        raise ValueError("draft_len, kept must have n entries and k_out one")
    if scores is not None and scores.numel() != k_max + 1:
        raise ValueError("scores must have k_max + 1 entries")
    _check(_lib.sv_uniform_k_select(_ptr(conf), _ptr(draft_len), n, k_max, _ptr(cost),
                                    cost.numel(), int(t_base), int(n_bonus), _ptr(kept),
                                    _ptr(k_out), _ptr(scores), _ptr(dev_error), _stream(stream)),
           "sv_uniform_k_select")


def sv_pack_varlen(kept, last_token, draft_tokens, cu_rows, row_req, row_pos, packed_tokens,
                   dev_error=None, stream=None):
    """kept [n], last_token [n], draft_tokens [n, k_max] -> cu_rows [n+1], row maps [n(k_max+1)]."""
    for name, t in (("kept", kept), ("last_token", last_token), ("cu_rows", cu_rows),
                    ("row_req", row_req), ("row_pos", row_pos), ("packed_tokens", packed_tokens)):
        _dev(t, torch.int32, name, 1)
    _dev(draft_tokens, torch.int32, "draft_tokens", 2)
    _dev(dev_error, torch.int32, "dev_error", 1)
    n, k_max = draft_tokens.shape
    cap = n * (k_max + 1)
    if kept.numel() != n or last_token.numel() != n or cu_rows.numel() != n + 1:
        raise ValueError("kept/last_token need n entries, cu_rows n+1")
    if row_req.numel() != cap or row_pos.numel() != cap or packed_tokens.numel() != cap:
        raise ValueError("row maps need n*(k_max+1) entries")
    _check(_lib.sv_pack_varlen(_ptr(kept), _ptr(last_token), _ptr(draft_tokens), n, k_max,
                               _ptr(cu_rows), _ptr(row_req), _ptr(row_pos), _ptr(packed_tokens),
                               _ptr(dev_error), _stream(stream)),
           "sv_pack_varlen")


_DTYPES = {torch.bfloat16: SV_BF16, torch.float32: SV_F32}


def _verify_args(target, draft, draft_tokens, cu_rows, mode, temperature, seed, step,
                 out_tokens, out_accepted, ws, out_p_draft, out_q_draft, out_residual_mass,
                 dev_error, vocab, out_q_entropy, out_q_max):
    if target.dtype not in _DTYPES:
        raise ValueError("logits must be bfloat16 or float32")
    _dev(target, target.dtype, "target", 2)
    if draft is not None:
        _dev(draft, target.dtype, "draft", 2)
    _dev(draft_tokens, torch.int32, "draft_tokens", 2)
    _dev(cu_rows, torch.int32, "cu_rows", 1)
    _dev(out_tokens, torch.int32, "out_tokens", 2)
    _dev(out_accepted, torch.int32, "out_accepted", 1)
    _dev(ws, torch.uint8, "ws", 1)
    for name, t in (("out_p_draft", out_p_draft), ("out_q_draft", out_q_draft),
                    ("out_q_entropy", out_q_entropy), ("out_q_max", out_q_max)):
        _dev(t, torch.float32, name, 2)
    _dev(out_residual_mass, torch.float32, "out_residual_mass", 1)
    _dev(dev_error, torch.int32, "dev_error", 1)
    n, k_max = draft_tokens.shape
    V = target.shape[1] if vocab is None else int(vocab)
    if cu_rows.numel() != n + 1 or tuple(out_tokens.shape) != (n, k_max + 1) \
            or out_accepted.numel() != n:
        raise ValueError("cu_rows [n+1], out_tokens [n, k_max+1], out_accepted [n]")
    if draft is not None and draft.shape[0] < n * k_max:
        raise ValueError("draft must hold n*k_max rows")
    for t in (out_p_draft, out_q_draft, out_q_entropy, out_q_max):
        if t is not None and tuple(t.shape) != (n, k_max):
            raise ValueError("out_p_draft, out_q_draft, out_q_entropy, out_q_max must be "
                             "[n, k_max]")
    if out_residual_mass is not None and out_residual_mass.numel() != n:
        raise ValueError("out_residual_mass must have n entries")
    return [_ptr(target), target.shape[1], target.shape[0], _ptr(draft),
            0 if draft is None else draft.shape[1], _DTYPES[target.dtype], V,
            _ptr(draft_tokens), _ptr(cu_rows), n, k_max, int(mode), float(temperature),
            int(seed), int(step), _ptr(out_tokens), _ptr(out_accepted), _ptr(out_p_draft),
            _ptr(out_q_draft), _ptr(out_residual_mass), _ptr(out_q_entropy), _ptr(out_q_max),
            _ptr(dev_error), _ptr(ws), 0 if ws is None else ws.numel()]


def sv_verify(target, draft, draft_tokens, cu_rows, mode, temperature, seed, step, out_tokens,
              out_accepted, ws, out_p_draft=None, out_q_draft=None, out_residual_mass=None,
              dev_error=None, vocab=None, stream=None, out_q_entropy=None, out_q_max=None):
    """target [rows, >=V] and draft [n*k_max, >=V] (bf16 or f32, row stride = shape[1]);
    draft_tokens [n, k_max] i32; cu_rows [n+1] i32; ws: uint8 device buffer of
    sv_verify_workspace_bytes(n, k_max) bytes; out_q_entropy / out_q_max [n, k_max] f32
    ask pass 1 for the draft-row features."""
    args = _verify_args(target, draft, draft_tokens, cu_rows, mode, temperature, seed, step,
                        out_tokens, out_accepted, ws, out_p_draft, out_q_draft,
                        out_residual_mass, dev_error, vocab, out_q_entropy, out_q_max)
    _check(_lib.sv_verify(*args, _stream(stream)), "sv_verify")


def sv_verify_stages(target, draft, draft_tokens, cu_rows, mode, temperature, seed, step,
                     out_tokens, out_accepted, ws, stages, out_p_draft=None, out_q_draft=None,
                     out_residual_mass=None, dev_error=None, vocab=None, stream=None,
                     out_q_entropy=None, out_q_max=None):
    """sv_verify restricted to pass 1 (stages=1), pass 2 (stages=2) or both (3)."""
    args = _verify_args(target, draft, draft_tokens, cu_rows, mode, temperature, seed, step,
                        out_tokens, out_accepted, ws, out_p_draft, out_q_draft,
                        out_residual_mass, dev_error, vocab, out_q_entropy, out_q_max)
    _check(_lib.sv_verify_stages(*args, int(stages), _stream(stream)), "sv_verify_stages")


def sv_verify_noalloc(target, draft, draft_tokens, cu_rows, mode, temperature, seed, step,
                      out_tokens, out_accepted, out_p_draft=None, out_q_draft=None,
                      out_residual_mass=None, dev_error=None, vocab=None, stream=None,
                      out_q_entropy=None, out_q_max=None):
    """sv_verify without a workspace argument: the library's static per-GPU array
    serves as the workspace (the call allocates nothing; overlapping calls on one
    GPU race on it)."""
    args = _verify_args(target, draft, draft_tokens, cu_rows, mode, temperature, seed, step,
                        out_tokens, out_accepted, None, out_p_draft, out_q_draft,
                        out_residual_mass, dev_error, vocab, out_q_entropy, out_q_max)
    _check(_lib.sv_verify_noalloc(*args[:-2], _stream(stream)), "sv_verify_noalloc")


def sv_accept_stats(accepted, cu_rows, attempted, accepted_at, totals, stream=None):
    """accepted [n] i32, cu_rows [n+1] i32 -> adds to attempted/accepted_at [k_max] and
    totals [2] (int64 device tensors holding uint64 counts)."""
    _dev(accepted, torch.int32, "accepted", 1)
    _dev(cu_rows, torch.int32, "cu_rows", 1)
    for name, t in (("attempted", attempted), ("accepted_at", accepted_at), ("totals", totals)):
        _dev(t, torch.int64, name, 1)
    n = accepted.numel()
    k_max = attempted.numel()
    if cu_rows.numel() != n + 1 or accepted_at.numel() != k_max or totals.numel() < 2:
        raise ValueError("cu_rows [n+1], attempted/accepted_at [k_max], totals [2]")
    _check(_lib.sv_accept_stats(_ptr(accepted), _ptr(cu_rows), n, k_max, _ptr(attempted),
                                _ptr(accepted_at), _ptr(totals), _stream(stream)),
           "sv_accept_stats")


def _features(q_draft, q_entropy, q_max):
    _dev(q_draft, torch.float32, "q_draft", 2)
    for name, t in (("q_entropy", q_entropy), ("q_max", q_max)):
        _dev(t, torch.float32, name, 2)
        if t is not None and t.shape != q_draft.shape:
            raise ValueError(f"{name} must have q_draft's shape")
    return q_draft.shape


def sv_calibrate_update(theta, q_draft, accepted, cu_rows, lr, count_out=None, stream=None,
                        q_entropy=None, q_max=None):
    """theta [k_max+3] f32 (in place); q_draft, q_entropy, q_max [n, k_max] f32 (the last
    two may be None: feature 0); accepted [n]; cu_rows [n+1]."""
    _dev(theta, torch.float32, "theta", 1)
    _dev(accepted, torch.int32, "accepted", 1)
    _dev(cu_rows, torch.int32, "cu_rows", 1)
    _dev(count_out, torch.int32, "count_out", 1)
    n, k_max = _features(q_draft, q_entropy, q_max)
    if theta.numel() != k_max + 3 or accepted.numel() != n or cu_rows.numel() != n + 1:
        raise ValueError("theta [k_max+3], accepted [n], cu_rows [n+1]")
    _check(_lib.sv_calibrate_update(_ptr(theta), _ptr(q_draft), _ptr(q_entropy), _ptr(q_max),
                                    _ptr(accepted), _ptr(cu_rows), n, k_max, float(lr),
                                    _ptr(count_out), _stream(stream)),
           "sv_calibrate_update")


def sv_calibrate_predict(theta, q_draft, conf, stream=None, q_entropy=None, q_max=None):
    """conf [n, k_max] f32 <- sigmoid(alpha_j + beta . x(q, entropy, max prob))."""
    _dev(theta, torch.float32, "theta", 1)
    _dev(conf, torch.float32, "conf", 2)
    n, k_max = _features(q_draft, q_entropy, q_max)
    if theta.numel() != k_max + 3 or tuple(conf.shape) != (n, k_max):
        raise ValueError("theta [k_max+3], conf [n, k_max]")
    _check(_lib.sv_calibrate_predict(_ptr(theta), _ptr(q_draft), _ptr(q_entropy), _ptr(q_max), n,
                                     k_max, _ptr(conf), _stream(stream)),
           "sv_calibrate_predict")


def sv_philox_uniforms(seed, step, u, v, stream=None):
    """u, v [n, n_pos] f32 <- the uniforms sv_verify draws for (r, j, step)."""
    _dev(u, torch.float32, "u", 2)
    _dev(v, torch.float32, "v", 2)
    n, n_pos = u.shape
    if tuple(v.shape) != (n, n_pos):
        raise ValueError("u and v must have the same shape")
    _check(_lib.sv_philox_uniforms(int(seed), int(step), n, n_pos, _ptr(u), _ptr(v),
                                   _stream(stream)),
           "sv_philox_uniforms")


class Sampling(NamedTuple):
    """Settings of truncated laws, one entry a row (sv_sample) or request
    (sv_verify_truncated), each a device tensor or None: temperature f32 (None: 1; 0: greedy),
    top_k i32 (None or <= 0: off), top_p f32 (None or >= 1: off), min_p f32 (None or 0: off)."""
    temperature: Optional[torch.Tensor] = None
    top_k: Optional[torch.Tensor] = None
    top_p: Optional[torch.Tensor] = None
    min_p: Optional[torch.Tensor] = None


def _law(law, n, device, name="law"):
    if law is None:
        return None
    n = (n,)
    return ctypes.byref(_Law(_on(law.temperature, torch.float32, f"{name}.temperature", device, n),
                             _on(law.top_k, torch.int32, f"{name}.top_k", device, n),
                             _on(law.top_p, torch.float32, f"{name}.top_p", device, n),
                             _on(law.min_p, torch.float32, f"{name}.min_p", device, n)))


def _logits(t, name, vocab):
    """(address, row stride, rows) of a logit matrix, whose rows may lie further apart than
    they are long."""
    if not t.is_cuda or t.dtype not in _DTYPES or t.dim() != 2:
        raise ValueError(f"{name} must be a bfloat16 or float32 device matrix")
    rows, width = t.shape
    if vocab is not None and vocab > width:
        raise ValueError(f"vocab must not pass {name}'s width")
    if t.is_contiguous():
        return t.data_ptr(), width, rows
    if width > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if rows > 1 and t.stride(0) < width:
        raise ValueError(f"{name}'s rows must not overlap")
    return t.data_ptr(), t.stride(0) if rows > 1 else width, rows


def sv_sample(logits, u, law, out_tokens, out_prob=None, out_support=None, dev_error=None,
              vocab=None, stream=None):
    """logits [rows, >=V] (bf16 or f32), u [rows] f32 in [0, 1) -> out_tokens [rows] i32 drawn
    under law (a Sampling or None), out_prob [rows] f32, out_support [rows] i32.
    u of drafts: not the uniforms of the (seed, step) that verifies them."""
    at, ld, n = _logits(logits, "logits", vocab)
    device, rows = logits.get_device(), (n,)
    _launch(_lib.sv_sample, "sv_sample", device, stream, at, ld, n, _DTYPES[logits.dtype],
            logits.shape[1] if vocab is None else int(vocab), _law(law, n, device),
            _on(u, torch.float32, "u", device, rows),
            _on(out_tokens, torch.int32, "out_tokens", device, rows),
            _on(out_prob, torch.float32, "out_prob", device, rows),
            _on(out_support, torch.int32, "out_support", device, rows),
            _on(dev_error, torch.int32, "dev_error", device, None))


def sv_verify_truncated_workspace_bytes(n_req, k_max):
    return int(_lib.sv_verify_truncated_workspace_bytes(n_req, k_max))


def sv_verify_truncated(target, draft, draft_tokens, cu_rows, target_law, draft_law, seed, step,
                        out_tokens, out_accepted, ws, out_p_draft=None, out_q_draft=None,
                        out_residual_mass=None, dev_error=None, vocab=None, stream=None):
    """sv_verify with each request's truncated laws: target [rows, >=V], draft [n*k_max, >=V]
    (None if k_max is 0), target_law and draft_law a Sampling of [n] settings or None;
    ws: uint8 device buffer of sv_verify_truncated_workspace_bytes(n, k_max) bytes."""
    at, ld, rows = _logits(target, "target", vocab)
    device = target.get_device()
    V = target.shape[1] if vocab is None else int(vocab)
    if draft_tokens.dim() != 2:
        raise ValueError("draft_tokens must have 2 dimensions")
    n, k_max = draft_tokens.shape
    draft_at, draft_ld = None, V
    if draft is not None:
        draft_at, draft_ld, draft_rows = _logits(draft, "draft", V)
        if draft.dtype is not target.dtype or draft_rows < n * k_max \
                or draft.get_device() != device:
            raise ValueError("draft must hold n*k_max rows of the target's type, on its device")
    _launch(_lib.sv_verify_truncated, "sv_verify_truncated", device, stream, at, ld, rows,
            draft_at, draft_ld, _DTYPES[target.dtype], V,
            _on(draft_tokens, torch.int32, "draft_tokens", device, None),
            _on(cu_rows, torch.int32, "cu_rows", device, (n + 1,)), n, k_max,
            _law(target_law, n, device, "target_law"), _law(draft_law, n, device, "draft_law"),
            int(seed), int(step), _on(out_tokens, torch.int32, "out_tokens", device, (n, k_max + 1)),
            _on(out_accepted, torch.int32, "out_accepted", device, (n,)),
            _on(out_p_draft, torch.float32, "out_p_draft", device, (n, k_max)),
            _on(out_q_draft, torch.float32, "out_q_draft", device, (n, k_max)),
            _on(out_residual_mass, torch.float32, "out_residual_mass", device, (n,)),
            _on(dev_error, torch.int32, "dev_error", device, None),
            _on(ws, torch.uint8, "ws", device, None), 0 if ws is None else ws.numel())


class TokenHistory:
    """What requests have said: counts [n_slots, vocab] i32, seen [n_slots, cap] i32, n_seen
    [n_slots] i32, as sv_history describes them (start with zeroed counts and n_seen).

    The tensors' addresses are taken once: they cannot be exchanged, and their storage must not
    be (set_, resize_)."""

    __slots__ = ("_counts", "_seen", "_n_seen", "_device", "_vocab", "_c", "_at")
    counts = property(lambda self: self._counts)
    seen = property(lambda self: self._seen)
    n_seen = property(lambda self: self._n_seen)
    device = property(lambda self: self._device)
    vocab = property(lambda self: self._vocab)

    def __init__(self, counts, seen, n_seen):
        if not counts.is_cuda or counts.dim() != 2 or seen.dim() != 2:
            raise ValueError("counts must be [n_slots, vocab] and seen [n_slots, cap] device tensors")
        self._counts, self._seen, self._n_seen = counts, seen, n_seen
        self._device = counts.get_device()
        n_slots, self._vocab = counts.shape
        cap = seen.shape[1]
        self._c = _History(_on(counts, torch.int32, "counts", self._device, None),
                           _on(seen, torch.int32, "seen", self._device, (n_slots, cap)),
                           _on(n_seen, torch.int32, "n_seen", self._device, (n_slots,)), n_slots,
                           self._vocab, cap)
        self._at = ctypes.addressof(self._c)

    @classmethod
    def empty(cls, n_slots, vocab, cap=None, device="cuda"):
        """A history of empty slots; cap: ids a slot lists (None: every id fits)."""
        return cls(torch.zeros(n_slots, vocab, dtype=torch.int32, device=device),
                   torch.zeros(n_slots, vocab if cap is None else cap, dtype=torch.int32,
                               device=device),
                   torch.zeros(n_slots, dtype=torch.int32, device=device))


def sv_history_clear(history, slots, dev_error=None, stream=None):
    """Empties the slots named by slots [n] i32."""
    device = history._device
    at = _on(slots, torch.int32, "slots", device, (slots.numel(),))
    _launch(_lib.sv_history_clear, "sv_history_clear", device, stream, history._at, at,
            slots.shape[0], _on(dev_error, torch.int32, "dev_error", device, None))


def sv_history_add(history, slots, tokens, in_prompt=False, dev_error=None, stream=None):
    """tokens [n, width] i32 (-1: skipped) added to slots [n] i32 (None: row r to slot r), as
    the prompt's ids or as emitted ones."""
    device = history._device
    if tokens.dim() != 2:
        raise ValueError("tokens must have 2 dimensions")
    n, width = tokens.shape
    ld = width
    if not tokens.is_contiguous():
        if tokens.dtype is not torch.int32 or tokens.get_device() != device \
                or (width > 1 and tokens.stride(1) != 1) or (n > 1 and tokens.stride(0) < width):
            raise ValueError("tokens must be int32 rows on the history's device")
        ld, at = (tokens.stride(0) if n > 1 else width), tokens.data_ptr()
    else:
        at = _on(tokens, torch.int32, "tokens", device, None)
    _launch(_lib.sv_history_add, "sv_history_add", device, stream, history._at,
            _on(slots, torch.int32, "slots", device, (n,)), at, ld, n, width, int(bool(in_prompt)),
            _on(dev_error, torch.int32, "dev_error", device, None))


class Penalties(NamedTuple):
    """Per-request penalties [n] f32, each a device tensor or None: repetition (None: 1),
    frequency (None: 0), presence (None: 0)."""
    repetition: Optional[torch.Tensor] = None
    frequency: Optional[torch.Tensor] = None
    presence: Optional[torch.Tensor] = None


class Bias(NamedTuple):
    """Per-request biases: request r's are entries start[r] .. start[r + 1] - 1 of ids (i32,
    ascending, each once) and values (f32, finite or -inf); start [n + 1] i32."""
    start: torch.Tensor
    ids: torch.Tensor
    values: torch.Tensor


class TokenMask(NamedTuple):
    """Allowed ids: bits [masks, >= ceil(vocab / 32)] i32 (id x: bit x % 32 of word x // 32),
    row_mask [rows] i32: each row's mask, -1: none (None: row i has mask i)."""
    bits: torch.Tensor
    row_mask: Optional[torch.Tensor] = None


def sv_adjust_logits(logits, out, row_req, row_pos, history=None, slots=None, penalties=None,
                     draft_tokens=None, bias=None, mask=None, dev_error=None, n_req=None,
                     stream=None):
    """logits [rows, V] (bf16 or f32) -> out (the same shape and type; out = logits: in place)
    under the requests' penalties, biases and grammar masks.  Row i is position row_pos[i] of
    request row_req[i] (-1: skipped; both None: row i is request i); the drafts before a row's
    position (draft_tokens [n, k_max] i32) count as said.  history, slots [n] i32: what was said
    before.  n_req: needed where no other argument tells it."""
    at, ld, rows = _logits(logits, "logits", None)
    out_at, out_ld, _ = _logits(out, "out", None)
    device, V = logits.get_device(), logits.shape[1]
    if out.shape != logits.shape or out.dtype is not logits.dtype or out.get_device() != device:
        raise ValueError("out must be of the logits' shape and type, on their device")
    k_max, drafts = 0, None
    if draft_tokens is not None:
        if draft_tokens.dim() != 2:
            raise ValueError("draft_tokens must have 2 dimensions")
        drafts = _on(draft_tokens, torch.int32, "draft_tokens", device, None)
        n, k_max = draft_tokens.shape
    elif n_req is not None:
        n = int(n_req)
    elif slots is not None:
        n = slots.shape[0]
    elif row_req is None:
        n = rows
    elif bias is not None:
        n = bias.start.shape[0] - 1
    else:
        raise ValueError("n_req is needed without draft_tokens, slots and bias")
    if n_req is not None and n != n_req:
        raise ValueError("draft_tokens must have n_req rows")
    if history is not None and history._device != device:
        raise ValueError("the history must be on the logits' device")
    pen = b = m = None
    if penalties is not None:
        pen = _Penalties(*(_on(x, torch.float32, f"penalties.{name}", device, (n,))
                           for name, x in zip(Penalties._fields, penalties)))
    if bias is not None:
        entries = bias.ids.numel()
        b = _Bias(_on(bias.start, torch.int32, "bias.start", device, (n + 1,)),
                  _on(bias.ids, torch.int32, "bias.ids", device, (entries,)),
                  _on(bias.values, torch.float32, "bias.values", device, (entries,)), entries)
    if mask is not None:
        bits = _on(mask.bits, torch.int32, "mask.bits", device, None)
        if mask.bits.dim() != 2:
            raise ValueError("mask.bits must have 2 dimensions")
        m = _TokenMask(bits, mask.bits.shape[1], mask.bits.shape[0],
                       _on(mask.row_mask, torch.int32, "mask.row_mask", device, (rows,)))
    _launch(_lib.sv_adjust_logits, "sv_adjust_logits", device, stream, at, ld, out_at, out_ld,
            rows, _DTYPES[logits.dtype], V, _on(row_req, torch.int32, "row_req", device, (rows,)),
            _on(row_pos, torch.int32, "row_pos", device, (rows,)), n, k_max, drafts,
            None if history is None else history._at,
            _on(slots, torch.int32, "slots", device, (n,)), _ref(pen), _ref(b), _ref(m),
            _on(dev_error, torch.int32, "dev_error", device, None))


def _ref(struct):
    return None if struct is None else ctypes.addressof(struct)


class PagedCache:
    """A paged key-value cache: k and v [n_pages, page_size, n_kv_heads, head_dim] (bfloat16 or
    float8_e4m3fn), any strides over pages, positions and heads that both share, the last
    dimension contiguous; k_scale, v_scale [n_kv_heads] f32 (float8 caches).

    The tensors' addresses and layout are taken once: they are held and cannot be exchanged
    (another cache is another PagedCache), and their storage must not be (set_, resize_)."""

    __slots__ = ("_k", "_v", "_k_scale", "_v_scale", "_device", "_n_kv_heads", "_head_dim",
                 "_page_size", "_c", "_at")
    k = property(lambda self: self._k)
    v = property(lambda self: self._v)
    k_scale = property(lambda self: self._k_scale)
    v_scale = property(lambda self: self._v_scale)
    device = property(lambda self: self._device)
    n_kv_heads = property(lambda self: self._n_kv_heads)
    head_dim = property(lambda self: self._head_dim)
    page_size = property(lambda self: self._page_size)

    def __init__(self, k, v, k_scale=None, v_scale=None):
        dtype = _CACHE_DTYPES.get(k.dtype)
        if not k.is_cuda or v.get_device() != k.get_device():
            raise ValueError("k and v must be device tensors on one device")
        if dtype is None or v.dtype is not k.dtype:
            raise ValueError("k and v must both be bfloat16 or float8_e4m3fn")
        strides = k.stride()
        if k.dim() != 4 or v.shape != k.shape or v.stride() != strides or strides[3] != 1:
            raise ValueError("k and v must be [n_pages, page_size, n_kv_heads, head_dim] with "
                             "the same strides, the last dimension contiguous")
        self._k, self._v, self._k_scale, self._v_scale = k, v, k_scale, v_scale
        self._device = k.get_device()
        n_pages, self._page_size, self._n_kv_heads, self._head_dim = k.shape
        if dtype == SV_BF16 and (k_scale is not None or v_scale is not None):
            raise ValueError("scales belong to float8 caches")
        heads = (self._n_kv_heads,)
        self._c = _Cache(k.data_ptr(), v.data_ptr(), dtype, n_pages, self._page_size,
                         self._n_kv_heads, self._head_dim, strides[0], strides[1], strides[2],
                         _on(k_scale, torch.float32, "k_scale", self._device, heads),
                         _on(v_scale, torch.float32, "v_scale", self._device, heads))
        self._at = ctypes.addressof(self._c)


_CACHE_DTYPES = {torch.bfloat16: SV_BF16, torch.float8_e4m3fn: SV_E4M3}


def _rows(t, name, device, heads, dim):
    """(address, row stride) of a [rows, heads, dim] bfloat16 tensor whose rows are contiguous."""
    if t.dtype is not torch.bfloat16 or t.get_device() != device or t.dim() != 3 \
            or t.shape[1] != heads or t.shape[2] != dim:
        raise ValueError(f"{name} must be bfloat16 [rows, {heads}, {dim}] on the cache's device")
    if t.is_contiguous():
        return t.data_ptr(), heads * dim
    if t.stride(2) != 1 or (heads > 1 and t.stride(1) != dim):
        raise ValueError(f"{name} must have contiguous heads within a row")
    return t.data_ptr(), t.stride(0) if t.shape[0] > 1 else heads * dim


def _table(page_table, device):
    at = _on(page_table, torch.int32, "page_table", device, None)
    if page_table.dim() != 2:
        raise ValueError("page_table must be [n, max_pages]")
    return at, page_table.shape[0], page_table.shape[1]


def sv_cache_append(cache, page_table, k, v, row_req, row_pos, ctx_len, dev_error=None,
                    stream=None):
    """Rows k, v [rows, n_kv_heads, head_dim] bf16 into the cache, row i at position
    ctx_len[row_req[i]] + row_pos[i] (the maps pack_varlen writes; -1: skipped);
    page_table [n, max_pages] i32, ctx_len [n] i32."""
    device = cache._device
    table, n, max_pages = _table(page_table, device)
    k_at, ld = _rows(k, "k", device, cache._n_kv_heads, cache._head_dim)
    v_at, v_ld = _rows(v, "v", device, cache._n_kv_heads, cache._head_dim)
    rows = k.shape[0]
    if v_ld != ld or v.shape[0] != rows:
        raise ValueError("k and v must have the same rows and row stride")
    _launch(_lib.sv_cache_append, "sv_cache_append", device, stream, cache._at, table, max_pages,
            k_at, v_at, ld, _on(row_req, torch.int32, "row_req", device, (rows,)),
            _on(row_pos, torch.int32, "row_pos", device, (rows,)), rows,
            _on(ctx_len, torch.int32, "ctx_len", device, (n,)), n,
            _on(dev_error, torch.int32, "dev_error", device, None))


def sv_cache_attend_workspace_bytes(n_req, k_max, n_heads, n_kv_heads, head_dim, max_pages,
                                    page_size):
    return int(_lib.sv_cache_attend_workspace_bytes(n_req, k_max, n_heads, n_kv_heads, head_dim,
                                                    max_pages, page_size))


def sv_cache_attend(cache, page_table, q, cu_rows, ctx_len, k_max, scale, out, ws=None,
                    out_lse=None, dev_error=None, stream=None):
    """Packed rows q [rows, n_heads, head_dim] bf16 -> out (same shape): row j of request r
    (packed row cu_rows[r] + j) sees the cache's positions 0 .. ctx_len[r] + j.
    ws: uint8 device buffer of sv_cache_attend_workspace_bytes(...) bytes (None if 0);
    out_lse [rows, n_heads] f32."""
    device = cache._device
    table, n, max_pages = _table(page_table, device)
    if q.dim() != 3 or out.shape != q.shape:
        raise ValueError("q must be [rows, n_heads, head_dim] and out of its shape")
    rows, heads, _ = q.shape
    q_at, q_ld = _rows(q, "q", device, heads, cache._head_dim)
    out_at, out_ld = _rows(out, "out", device, heads, cache._head_dim)
    _launch(_lib.sv_cache_attend, "sv_cache_attend", device, stream, cache._at, table, max_pages,
            q_at, q_ld, rows, heads, _on(cu_rows, torch.int32, "cu_rows", device, (n + 1,)),
            _on(ctx_len, torch.int32, "ctx_len", device, (n,)), n, int(k_max), float(scale),
            out_at, out_ld, _on(out_lse, torch.float32, "out_lse", device, (rows, heads)),
            _on(dev_error, torch.int32, "dev_error", device, None),
            _on(ws, torch.uint8, "ws", device, None), 0 if ws is None else ws.numel())


def sv_cache_attend_shared_workspace_bytes(n_req, n_groups, k_max, n_heads, n_kv_heads, head_dim,
                                           max_pages, page_size):
    return int(_lib.sv_cache_attend_shared_workspace_bytes(n_req, n_groups, k_max, n_heads,
                                                           n_kv_heads, head_dim, max_pages,
                                                           page_size))


def sv_cache_attend_shared(cache, page_table, q, cu_rows, ctx_len, group_start, prefix_len, k_max,
                           scale, out, ws, out_lse=None, dev_error=None, stream=None):
    """sv_cache_attend of a batch in groups of neighbours that share a prefix: requests
    group_start[g] .. group_start[g + 1] - 1 (group_start [groups + 1] i32) have their first
    prefix_len[g] positions ([groups] i32) in common, which are read once.
    ws: uint8 device buffer of sv_cache_attend_shared_workspace_bytes(...) bytes."""
    device = cache._device
    table, n, max_pages = _table(page_table, device)
    if q.dim() != 3 or out.shape != q.shape:
        raise ValueError("q must be [rows, n_heads, head_dim] and out of its shape")
    rows, heads, _ = q.shape
    groups = prefix_len.numel()
    q_at, q_ld = _rows(q, "q", device, heads, cache._head_dim)
    out_at, out_ld = _rows(out, "out", device, heads, cache._head_dim)
    _launch(_lib.sv_cache_attend_shared, "sv_cache_attend_shared", device, stream, cache._at, table,
            max_pages, q_at, q_ld, rows, heads, _on(cu_rows, torch.int32, "cu_rows", device, (n + 1,)),
            _on(ctx_len, torch.int32, "ctx_len", device, (n,)), n, int(k_max),
            _on(group_start, torch.int32, "group_start", device, (groups + 1,)),
            _on(prefix_len, torch.int32, "prefix_len", device, (groups,)), groups, float(scale),
            out_at, out_ld, _on(out_lse, torch.float32, "out_lse", device, (rows, heads)),
            _on(dev_error, torch.int32, "dev_error", device, None),
            _on(ws, torch.uint8, "ws", device, None), 0 if ws is None else ws.numel())


class LatentCache:
    """A paged cache of latent vectors: kv [n_pages, page_size, latent_dim + 64] (bfloat16 or
    float8_e4m3fn), any strides over pages and positions, the last dimension contiguous;
    latent_dim 256 or 512; scale [1] f32 (float8 caches).

    The tensor's address and layout are taken once: it is held and cannot be exchanged, and its
    storage must not be (set_, resize_)."""

    __slots__ = ("_kv", "_scale", "_device", "_latent_dim", "_page_size", "_c", "_at")
    kv = property(lambda self: self._kv)
    scale = property(lambda self: self._scale)
    device = property(lambda self: self._device)
    latent_dim = property(lambda self: self._latent_dim)
    page_size = property(lambda self: self._page_size)

    def __init__(self, kv, latent_dim, scale=None):
        dtype = _CACHE_DTYPES.get(kv.dtype)
        if not kv.is_cuda or dtype is None:
            raise ValueError("kv must be a bfloat16 or float8_e4m3fn device tensor")
        if kv.dim() != 3 or kv.stride(2) != 1 or kv.shape[2] != latent_dim + SV_LATENT_ROPE:
            raise ValueError("kv must be [n_pages, page_size, latent_dim + 64], the last dimension "
                             "contiguous")
        if dtype == SV_BF16 and scale is not None:
            raise ValueError("scales belong to float8 caches")
        self._kv, self._scale, self._device = kv, scale, kv.get_device()
        n_pages, self._page_size, _ = kv.shape
        self._latent_dim = int(latent_dim)
        self._c = _LatentCache(kv.data_ptr(), dtype, n_pages, self._page_size, self._latent_dim,
                               kv.stride(0), kv.stride(1),
                               _on(scale, torch.float32, "scale", self._device, (1,)))
        self._at = ctypes.addressof(self._c)


def _matrix(t, name, device, width):
    """(address, row stride) of a [rows, width] bfloat16 tensor whose rows are contiguous."""
    if t.dtype is not torch.bfloat16 or t.get_device() != device or t.dim() != 2 \
            or t.shape[1] != width:
        raise ValueError(f"{name} must be bfloat16 [rows, {width}] on the cache's device")
    if t.is_contiguous():
        return t.data_ptr(), width
    if t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    return t.data_ptr(), t.stride(0) if t.shape[0] > 1 else width


def sv_latent_append(cache, page_table, latent, rope, row_req, row_pos, ctx_len, dev_error=None,
                     stream=None):
    """Rows latent [rows, latent_dim] and rope [rows, 64] bf16 into the cache, row i at position
    ctx_len[row_req[i]] + row_pos[i] (the maps pack_varlen writes; -1: skipped);
    page_table [n, max_pages] i32, ctx_len [n] i32."""
    device = cache._device
    table, n, max_pages = _table(page_table, device)
    at, ld = _matrix(latent, "latent", device, cache._latent_dim)
    rope_at, rope_ld = _matrix(rope, "rope", device, SV_LATENT_ROPE)
    rows = latent.shape[0]
    if rope.shape[0] != rows:
        raise ValueError("latent and rope must have the same rows")
    _launch(_lib.sv_latent_append, "sv_latent_append", device, stream, cache._at, table, max_pages,
            at, ld, rope_at, rope_ld, _on(row_req, torch.int32, "row_req", device, (rows,)),
            _on(row_pos, torch.int32, "row_pos", device, (rows,)), rows,
            _on(ctx_len, torch.int32, "ctx_len", device, (n,)), n,
            _on(dev_error, torch.int32, "dev_error", device, None))


def sv_latent_attend_workspace_bytes(n_req, k_max, n_heads, latent_dim, max_pages, page_size):
    return int(_lib.sv_latent_attend_workspace_bytes(n_req, k_max, n_heads, latent_dim, max_pages,
                                                     page_size))


def sv_latent_attend(cache, page_table, q, cu_rows, ctx_len, k_max, scale, out, ws=None,
                     out_lse=None, dev_error=None, stream=None):
    """Packed rows q [rows, n_heads, latent_dim + 64] bf16 -> out [rows, n_heads, latent_dim]: row
    j of request r (packed row cu_rows[r] + j) sees the cache's positions 0 .. ctx_len[r] + j.
    ws: uint8 device buffer of sv_latent_attend_workspace_bytes(...) bytes (None if 0);
    out_lse [rows, n_heads] f32."""
    device, dim = cache._device, cache._latent_dim
    table, n, max_pages = _table(page_table, device)
    if q.dim() != 3 or out.dim() != 3 or out.shape[:2] != q.shape[:2]:
        raise ValueError("q must be [rows, n_heads, latent_dim + 64] and out [rows, n_heads, "
                         "latent_dim]")
    rows, heads, _ = q.shape
    q_at, q_ld = _rows(q, "q", device, heads, dim + SV_LATENT_ROPE)
    out_at, out_ld = _rows(out, "out", device, heads, dim)
    _launch(_lib.sv_latent_attend, "sv_latent_attend", device, stream, cache._at, table, max_pages,
            q_at, q_ld, rows, heads, _on(cu_rows, torch.int32, "cu_rows", device, (n + 1,)),
            _on(ctx_len, torch.int32, "ctx_len", device, (n,)), n, int(k_max), float(scale),
            out_at, out_ld, _on(out_lse, torch.float32, "out_lse", device, (rows, heads)),
            _on(dev_error, torch.int32, "dev_error", device, None),
            _on(ws, torch.uint8, "ws", device, None), 0 if ws is None else ws.numel())


# ----------------------------------------------------------------------------
# Allocating conveniences over the calls above (outputs are new device tensors).

def budget_select(conf, draft_len, cost, t_base, n_bonus, stream=None):
    dev = conf.device
    n, k_max = conf.shape
    kept = torch.empty(n, dtype=torch.int32, device=dev)
    budget = torch.empty(1, dtype=torch.int32, device=dev)
    survival = torch.empty(n, k_max, dtype=torch.float32, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    ws = torch.empty(max(1, sv_budget_workspace_bytes(n, k_max)), dtype=torch.uint8, device=dev)
    sv_budget_select(conf, draft_len, cost, t_base, n_bonus, kept, budget, survival, err, stream,
                     ws=ws)
    return dict(kept=kept, budget=budget, survival=survival, dev_error=err)


def budget_allocate(conf, draft_len, budget_in, stream=None, ws=None):
    dev = conf.device
    n, k_max = conf.shape
    out = dict(kept=torch.empty(n, dtype=torch.int32, device=dev),
               budget_used=torch.empty(1, dtype=torch.int32, device=dev),
               survival=torch.empty(n, k_max, dtype=torch.float32, device=dev),
               dev_error=torch.zeros(1, dtype=torch.int32, device=dev))
    if ws is None:
        ws = torch.empty(max(1, sv_budget_workspace_bytes(n, k_max)), dtype=torch.uint8,
                         device=dev)
    sv_budget_allocate(conf, draft_len, budget_in, out["kept"], out["budget_used"],
                       out["survival"], out["dev_error"], stream, ws=ws)
    return out


def uniform_k_select(conf, draft_len, cost, t_base, n_bonus, stream=None):
    dev = conf.device
    n, k_max = conf.shape
    out = dict(kept=torch.empty(n, dtype=torch.int32, device=dev),
               k=torch.empty(1, dtype=torch.int32, device=dev),
               scores=torch.empty(k_max + 1, dtype=torch.float64, device=dev),
               dev_error=torch.zeros(1, dtype=torch.int32, device=dev))
    sv_uniform_k_select(conf, draft_len, cost, t_base, n_bonus, out["kept"], out["k"],
                        out["scores"], out["dev_error"], stream)
    return out


def pack_varlen(kept, last_token, draft_tokens, stream=None):
    dev = kept.device
    n, k_max = draft_tokens.shape
    cap = n * (k_max + 1)
    out = dict(cu_rows=torch.empty(n + 1, dtype=torch.int32, device=dev),
               row_req=torch.empty(cap, dtype=torch.int32, device=dev),
               row_pos=torch.empty(cap, dtype=torch.int32, device=dev),
               packed_tokens=torch.empty(cap, dtype=torch.int32, device=dev),
               dev_error=torch.zeros(1, dtype=torch.int32, device=dev))
    sv_pack_varlen(kept, last_token, draft_tokens, out["cu_rows"], out["row_req"],
                   out["row_pos"], out["packed_tokens"], out["dev_error"], stream)
    return out


def verify(target, draft, draft_tokens, cu_rows, mode, temperature=1.0, seed=0, step=0,
           vocab=None, stream=None, stages=None, ws=None, features=False):
    """Allocating wrapper: sv_verify, or sv_verify_stages(stages) when `stages` is given.
    ws: a workspace to reuse.  features: also return the draft-row features q_entropy and
    q_max (pass 1 then accumulates them)."""
    dev = target.device
    n, k_max = draft_tokens.shape
    if ws is None:
        ws = torch.zeros(max(1, sv_verify_workspace_bytes(n, k_max)), dtype=torch.uint8,
                         device=dev)
    out = dict(tokens=torch.empty(n, k_max + 1, dtype=torch.int32, device=dev),
               accepted=torch.empty(n, dtype=torch.int32, device=dev),
               p_draft=torch.empty(n, k_max, dtype=torch.float32, device=dev),
               q_draft=torch.empty(n, k_max, dtype=torch.float32, device=dev),
               residual_mass=torch.empty(n, dtype=torch.float32, device=dev),
               dev_error=torch.zeros(1, dtype=torch.int32, device=dev))
    if features:
        out["q_entropy"] = torch.empty(n, k_max, dtype=torch.float32, device=dev)
        out["q_max"] = torch.empty(n, k_max, dtype=torch.float32, device=dev)
    feat = dict(out_q_entropy=out.get("q_entropy"), out_q_max=out.get("q_max"))
    if stages is None:
        sv_verify(target, draft, draft_tokens, cu_rows, mode, temperature, seed, step,
                  out["tokens"], out["accepted"], ws, out["p_draft"], out["q_draft"],
                  out["residual_mass"], out["dev_error"], vocab, stream, **feat)
    else:
        sv_verify_stages(target, draft, draft_tokens, cu_rows, mode, temperature, seed, step,
                         out["tokens"], out["accepted"], ws, stages, out["p_draft"],
                         out["q_draft"], out["residual_mass"], out["dev_error"], vocab, stream,
                         **feat)
    return out
