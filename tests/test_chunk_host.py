"""Chunk attention's entry points on the host: every refusal comes before anything is
launched.  No compute call is made here."""
import ctypes

import pytest

import fp8_paged_attention_e4m3_gb300 as vae4

FAKE = 0x100000  # never dereferenced: every case below fails validation or has no work
U8, I32, F16, F32, BF16 = vae4.VAE4_U8, vae4.VAE4_I32, vae4.VAE4_F16, vae4.VAE4_F32, 5
B, Q, HQ, HKV, D, PAGE, NB, NPG, MP = 3, 40, 6, 2, 128, 96, 2, 40, 16
NULL, DTYPE, SHAPE, STRIDE, ALIGN, UNSUP, WS = -1, -2, -3, -4, -5, -6, -8
ORDER = ("q", "k", "v", "bt", "seq", "sc", "out", "ws")


@pytest.fixture(scope="module")
def lib():
    return vae4.load()


def _t(dtype, shape, strides=None, data=FAKE):
    d = vae4.Tensor()
    d.data, d.dtype, d.ndim = data, dtype, len(shape)
    if strides is None:
        strides, acc = [], 1
        for s in reversed(shape):
            strides.insert(0, acc)
            acc *= s
    for k, (s, st) in enumerate(zip(shape, strides)):
        d.shape[k], d.stride[k] = s, st
    return d


def base():
    return dict(q=_t(F16, [B, Q, HQ, D]), k=_t(U8, [NPG, PAGE, HKV, D]), v=_t(U8, [NPG, PAGE, HKV, D]),
                bt=_t(I32, [B, MP]), seq=_t(I32, [B, 2]), sc=_t(F32, [NPG, 2, HKV, NB]),
                out=_t(F16, [B, Q, HQ, D]), ws=_t(U8, [1 << 30]))


def call(lib, a, **opt):
    o = vae4.Options(opt.get("scale", 0.0), opt.get("part", 0), opt.get("cap", 0), opt.get("sms", 152),
                     opt.get("flags", 0), opt.get("hilo", 0))
    return lib.verify_attn_e4m3_chunk(*[ctypes.byref(a[k]) if a[k] is not None else None for k in ORDER], None,
                                      ctypes.byref(o))


@pytest.mark.parametrize("over,code", [
    (dict(q=_t(F32, [B, Q, HQ, D])), DTYPE),
    (dict(q=_t(BF16, [B, Q, HQ, D])), DTYPE),  # out is of another type
    (dict(k=_t(F16, [NPG, PAGE, HKV, D])), DTYPE),
    (dict(bt=_t(F32, [B, MP])), DTYPE),
    (dict(seq=_t(F32, [B, 2])), DTYPE),
    (dict(sc=_t(F16, [NPG, 2, HKV, NB])), DTYPE),
    (dict(sc=_t(F16, [HKV, 2])), DTYPE),
    (dict(ws=_t(F32, [1 << 28])), DTYPE),
    (dict(q=_t(F16, [B, Q, HQ])), SHAPE),
    (dict(out=_t(F16, [B, Q + 1, HQ, D])), SHAPE),
    (dict(v=_t(U8, [NPG, PAGE, HKV + 1, D])), SHAPE),
    (dict(bt=_t(I32, [B + 1, MP])), SHAPE),
    (dict(seq=_t(I32, [B, 3])), SHAPE),
    (dict(sc=_t(F32, [HKV + 1, 2])), SHAPE),
    (dict(sc=_t(F32, [NPG, 2, HKV, 5])), UNSUP),
    (dict(q=_t(F16, [B, 65537, HQ, D]), out=_t(F16, [B, 65537, HQ, D])), SHAPE),
    (dict(q=_t(F16, [B, Q, 7, D]), out=_t(F16, [B, Q, 7, D])), -7),  # heads that no KV heads divide
    (dict(q=_t(F16, [B, Q, HQ, 96]), out=_t(F16, [B, Q, HQ, 96]), k=_t(U8, [NPG, PAGE, HKV, 96]),
          v=_t(U8, [NPG, PAGE, HKV, 96])), UNSUP),
    (dict(q=_t(F16, [B, Q, HQ, D], [Q * HQ * D, HQ * D, D, 2])), STRIDE),
    (dict(q=_t(F16, [B, Q, HQ, D], [Q * HQ * D, HQ * D, D + 4, 1])), STRIDE),
    (dict(out=_t(F16, [B, Q, HQ, D], [Q * HQ * D, HQ * D, 0, 1])), STRIDE),  # heads in one place
    (dict(sc=_t(F32, [HKV, 2], [2, 2])), STRIDE),
    (dict(q=_t(F16, [B, Q, HQ, D], data=FAKE + 8)), ALIGN),
    (dict(sc=_t(F32, [HKV, 2], data=FAKE + 2)), ALIGN),
    (dict(ws=_t(U8, [4096])), WS),
    (dict(ws=_t(U8, [1 << 30], data=FAKE + 64)), WS),
])
def test_refusals(lib, over, code):
    a = base()
    a.update(over)
    assert call(lib, a) == code


def test_null_tensors_and_pointers(lib):
    for k in ORDER:
        a = base()
        a[k] = None
        assert call(lib, a) == NULL, k
        a = base()
        a[k].data = None
        assert call(lib, a) == NULL, k


def test_options(lib):
    a = base()
    assert call(lib, a, flags=vae4.FLAG_WARP_MMA) == UNSUP and call(lib, a, hilo=1) == UNSUP
    assert call(lib, a, part=64) == vae4_code("PARTITION") and call(lib, a, cap=MP * PAGE + 1) == SHAPE
    for bad in (dict(flags=1 << 20), dict(hilo=2), dict(scale=-1.0), dict(scale=float("nan"))):
        assert call(lib, a, **bad) == vae4_code("OPTIONS")


def vae4_code(name):
    import os
    import re
    text = open(os.path.join(os.path.dirname(__file__), "..", "include", "verify_attn_e4m3.h")).read()
    return int(re.search(r"VAE4_ERR_%s\s*=\s*(-\d+)" % name, text)[1])


def test_no_sequences_is_no_error(lib):
    a = base()
    a.update(q=_t(F16, [0, Q, HQ, D], data=None), out=_t(F16, [0, Q, HQ, D], data=None),
             bt=_t(I32, [0, MP], data=None), seq=_t(I32, [0, 2], data=None))
    assert call(lib, a) == 0


def test_workspace_bytes_and_sizes_past_63_bits():
    n = vae4.chunk_workspace_bytes
    assert n(1, 1, 1, 1, 64, 128, 152) < n(8, 64, 8, 8192, 128, 8192, 152) <= n(64, 64, 8, 8192, 128, 1 << 20, 152)
    assert n(1, 512, 1, 65536, 64, 1 << 29, 152) > 0
    for bad in ((0, 1, 1, 1, 64, 128), (1, 1, 1, 1, 64, 0), (1, 1, 1, 65537, 64, 128), (1, 3, 2, 1, 64, 128),
                (1, 2048, 1, 1, 64, (1 << 30) - 1),               # a unit's places times its tiles
                (65535, 4096, 128, 65536, 64, 1 << 27)):          # the batch's places
        with pytest.raises(vae4.Vae4Error):
            n(*bad, 152)
