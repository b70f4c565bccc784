"""Host validation of the history and logit calls (CPU): refusals come before
anything is launched, and the binding refuses what does not fit."""

import ctypes

import pytest
import torch

sv = pytest.importorskip("adaptive_draft_verification_amd",
                         reason="libspecverify.so not built (python adaptive_draft_verification_amd/build.py)")

FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: every call below fails validation first
FAR = ctypes.c_void_p(0x900000)
ODD = ctypes.c_void_p(0x1001)


def history(**kw):
    args = dict(counts=0x1000, seen=0x2000, n_seen=0x3000, n_slots=4, vocab=64, cap=8)
    args.update(kw)
    return ctypes.byref(sv._History(*args.values()))


def clear(h=None, **kw):
    args = dict(slots=FAKE, n=2, dev_error=None, stream=None)
    args.update(kw)
    return sv._lib.sv_history_clear(history() if h is None else h, *args.values())


def add(h=None, **kw):
    args = dict(slots=FAKE, tokens=FAKE, ld=8, n=2, width=8, in_prompt=0, dev_error=None,
                stream=None)
    args.update(kw)
    return sv._lib.sv_history_add(history() if h is None else h, *args.values())


def adjust(**kw):
    args = dict(logits=FAKE, ld=64, out=FAR, out_ld=64, n_rows=4, dtype=sv.SV_BF16, vocab=64,
                row_req=FAKE, row_pos=FAKE, n_req=2, k_max=3, drafts=FAKE, history=history(),
                slots=None, penalties=ctypes.byref(sv._Penalties()), bias=None, mask=None,
                dev_error=None, stream=None)
    args.update(kw)
    return sv._lib.sv_adjust_logits(*args.values())


@pytest.mark.parametrize("kw", [dict(n_slots=-1), dict(vocab=0), dict(vocab=2 ** 20 + 1),
                                dict(cap=-1)])
def test_history_shapes(kw):
    assert clear(history(**kw)) == sv.SV_ERR_SHAPE
    assert add(history(**kw)) == sv.SV_ERR_SHAPE
    assert adjust(history=history(**kw)) == sv.SV_ERR_SHAPE


def test_history_refusals():
    none = ctypes.c_void_p(None)
    assert clear(none) == add(none) == sv.SV_ERR_NULL
    for kw in (dict(counts=None), dict(seen=None), dict(n_seen=None)):
        assert clear(history(**kw)) == add(history(**kw)) == sv.SV_ERR_NULL, kw
        assert adjust(history=history(**kw)) == sv.SV_ERR_NULL, kw
    for kw in (dict(n=-1), dict(n=sv.SV_MAX_HISTORY_TOKENS // 1024 + 1)):
        assert clear(**kw) == sv.SV_ERR_SHAPE, kw
    for kw in (dict(n=-1), dict(width=-1), dict(ld=7), dict(n=2 ** 22 + 1),
               dict(width=2 ** 30, ld=2 ** 30), dict(ld=2 ** 61)):
        assert add(**kw) == sv.SV_ERR_SHAPE, kw
    assert add(tokens=None) == sv.SV_ERR_NULL
    assert clear(n=0) == add(n=0, tokens=None) == add(width=0, tokens=None) == sv.SV_OK
    assert sv.SV_MAX_HISTORY_TOKENS < 2 ** 32


def test_adjust_refusals():
    assert adjust(dtype=sv.SV_E4M3) == adjust(dtype=9) == sv.SV_ERR_DTYPE
    for kw in (dict(n_rows=-1), dict(n_rows=sv.SV_MAX_SAMPLE_ROWS + 1), dict(vocab=0),
               dict(vocab=2 ** 20 + 1, ld=2 ** 21, out_ld=2 ** 21), dict(ld=63), dict(out_ld=63),
               dict(n_req=-1), dict(k_max=-1), dict(k_max=65), dict(history=history(vocab=63)),
               dict(logits=ODD), dict(out=ODD), dict(ld=2 ** 60), dict(out_ld=2 ** 60),
               dict(row_req=None, row_pos=None, n_rows=3, n_req=2),
               dict(out=ctypes.c_void_p(0x1000 + 64)), dict(out=ctypes.c_void_p(0x1000 - 64)),
               dict(out=FAKE, out_ld=65),
               dict(bias=ctypes.byref(sv._Bias(0x1000, 0x1000, 0x1000, -1))),
               dict(mask=ctypes.byref(sv._TokenMask(0x1000, 1, 1, None))),
               dict(mask=ctypes.byref(sv._TokenMask(0x1000, 2, -1, None)))):
        assert adjust(**kw) == sv.SV_ERR_SHAPE, kw
    for kw in (dict(logits=None), dict(out=None), dict(row_req=None), dict(row_pos=None),
               dict(drafts=None), dict(bias=ctypes.byref(sv._Bias(None, 0x1000, 0x1000, 1))),
               dict(bias=ctypes.byref(sv._Bias(0x1000, None, 0x1000, 1))),
               dict(bias=ctypes.byref(sv._Bias(0x1000, 0x1000, None, 1))),
               dict(mask=ctypes.byref(sv._TokenMask(None, 2, 1, None)))):
        assert adjust(**kw) == sv.SV_ERR_NULL, kw
    assert adjust(n_rows=0, logits=None, out=None) == sv.SV_OK
    assert sv.SV_DEV_BAD_SLOT == 512


def test_binding_refuses_host_tensors():
    z, i = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        sv.sv_adjust_logits(z, z, None, None)
    with pytest.raises(ValueError):
        sv.TokenHistory(i[:, None], i[:, None], i)


@pytest.mark.parametrize("name", ["counts", "seen", "n_seen", "device", "vocab"])
def test_history_fields_cannot_be_exchanged(name):
    with pytest.raises(AttributeError):
        setattr(object.__new__(sv.TokenHistory), name, None)
