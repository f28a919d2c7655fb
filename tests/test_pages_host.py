"""The pages' entry points on the host: every refusal comes before anything is
launched.  No compute call is made here."""
import ctypes

import pytest

import fp8_paged_attention_e4m3_gb300 as vae4

FAKE = 0x100000  # never dereferenced: every case below fails validation or has no work
U8, I32, F16, F32 = vae4.VAE4_U8, vae4.VAE4_I32, vae4.VAE4_F16, vae4.VAE4_F32
B, HKV, D, PAGE, NB, NPG, MP, N = 3, 2, 128, 96, 2, 40, 16, 5
NULL, DTYPE, SHAPE, STRIDE, ALIGN, UNSUP, WS = -1, -2, -3, -4, -5, -6, -8


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
    return dict(k=_t(U8, [NPG, PAGE, HKV, D]), v=_t(U8, [NPG, PAGE, HKV, D]), pairs=_t(I32, [N, 2]),
                sc=_t(F32, [NPG, 2, HKV, NB]), bd=_t(U8, [NPG, HKV, NB, 2, D]), bt=_t(I32, [B, MP]),
                rc=_t(I32, [NPG]), par=_t(I32, [B]), seq=_t(I32, [B, 2]), cp=_t(I32, [B, 2]),
                ws=_t(U8, [1 << 16]), mv=_t(I32, [N, 2]))


NEEDS = {"copy": ("k", "v", "pairs", "sc", "bd"), "fork": ("bt", "rc", "par"),
         "resize": ("bt", "seq", "rc", "cp", "ws"), "compact": ("bt", "rc", "mv")}
POOL = ("fork", "resize", "compact")


def call(lib, name, a, page=PAGE):
    r = [ctypes.byref(a[k]) if a[k] is not None else None for k in NEEDS[name]]
    if name == "resize":
        r.append(page)
    return getattr(lib, f"verify_attn_e4m3_{name}_pages")(*r, None, None)


@pytest.mark.parametrize("names,over,code", [
    # types
    (("copy",), dict(k=_t(F16, [NPG, PAGE, HKV, D])), DTYPE),
    (("copy",), dict(v=_t(F32, [NPG, PAGE, HKV, D])), DTYPE),
    (("copy",), dict(pairs=_t(F32, [N, 2])), DTYPE),
    (("copy",), dict(sc=_t(F16, [NPG, 2, HKV, NB])), DTYPE),
    (("copy",), dict(bd=_t(F16, [NPG, HKV, NB, 2, D])), DTYPE),
    (POOL, dict(bt=_t(F32, [B, MP])), DTYPE),
    (POOL, dict(rc=_t(F32, [NPG])), DTYPE),
    (("fork",), dict(par=_t(F32, [B])), DTYPE),
    (("resize",), dict(seq=_t(F32, [B, 2])), DTYPE),
    (("resize",), dict(cp=_t(F32, [B, 2])), DTYPE),
    (("resize",), dict(ws=_t(F32, [4096])), DTYPE),
    (("compact",), dict(mv=_t(F32, [N, 2])), DTYPE),
    # shapes
    (("copy",), dict(v=_t(U8, [NPG + 1, PAGE, HKV, D])), SHAPE),
    (("copy",), dict(k=_t(U8, [NPG, PAGE, D])), SHAPE),
    (("copy",), dict(pairs=_t(I32, [N, 3])), SHAPE),
    (("copy",), dict(pairs=_t(I32, [N])), SHAPE),
    (("copy",), dict(sc=_t(F32, [HKV, 2])), SHAPE),
    (("copy",), dict(sc=_t(F32, [NPG + 1, 2, HKV, NB])), SHAPE),
    (("copy",), dict(bd=_t(U8, [NPG, HKV, 1, 2, D])), SHAPE),
    (POOL, dict(bt=_t(I32, [B * MP])), SHAPE),
    (POOL, dict(bt=_t(I32, [B, 0])), SHAPE),
    (POOL, dict(bt=_t(I32, [1 << 20, 1 << 20])), SHAPE),
    (POOL, dict(rc=_t(I32, [0])), SHAPE),
    (POOL, dict(rc=_t(I32, [NPG, 1])), SHAPE),
    (POOL, dict(rc=_t(I32, [(1 << 30) + 1])), SHAPE),
    (("fork",), dict(par=_t(I32, [B + 1])), SHAPE),
    (("fork",), dict(bt=_t(I32, [8193, 2]), par=_t(I32, [8193])), SHAPE),
    (("resize",), dict(seq=_t(I32, [B, 3])), SHAPE),
    (("resize",), dict(seq=_t(I32, [B + 1])), SHAPE),
    (("resize",), dict(cp=_t(I32, [B + 1, 2])), SHAPE),
    (("resize",), dict(bt=_t(I32, [16385, 2]), seq=_t(I32, [16385, 2]), cp=_t(I32, [16385, 2])), SHAPE),
    (("resize",), dict(bt=_t(I32, [B, 1 << 24])), SHAPE),  # past 2^30 tokens
    (("compact",), dict(mv=_t(I32, [N, 1])), SHAPE),
    # pages, blocks
    (("copy",), dict(k=_t(U8, [NPG, 24, HKV, D]), v=_t(U8, [NPG, 24, HKV, D])), UNSUP),
    (("copy",), dict(k=_t(U8, [NPG, PAGE, HKV, 96]), v=_t(U8, [NPG, PAGE, HKV, 96])), UNSUP),
    (("copy",), dict(sc=_t(F32, [NPG, 2, HKV, 5])), UNSUP),
    (("copy",), dict(sc=None, bd=_t(U8, [NPG, HKV, 5, 2, D])), UNSUP),
    # strides, rows that share memory, alignment
    (("copy",), dict(k=_t(U8, [NPG, PAGE, HKV, D], [0, HKV * D, D, 1])), STRIDE),
    (("copy",), dict(k=_t(U8, [NPG, PAGE, HKV, D], [PAGE * HKV * D, HKV * D, D + 4, 1])), STRIDE),
    (("copy",), dict(sc=_t(F32, [NPG, 2, HKV, NB], [2 * HKV * NB, 0, NB, 1])), STRIDE),
    (("copy",), dict(bd=_t(U8, [NPG, HKV, NB, 2, D], [0, 4 * D, 2 * D, D, 1])), STRIDE),
    (("copy",), dict(pairs=_t(I32, [N, 2], [1, N])), STRIDE),
    (POOL, dict(bt=_t(I32, [B, MP], [0, 1])), STRIDE),
    (POOL, dict(bt=_t(I32, [B, MP], [MP - 1, 1])), STRIDE),
    (POOL, dict(bt=_t(I32, [B, MP], [1, B])), STRIDE),
    (POOL, dict(rc=_t(I32, [NPG], [2])), STRIDE),
    (("fork",), dict(par=_t(I32, [B], [2])), STRIDE),
    (("resize",), dict(seq=_t(I32, [B, 2], [1, B])), STRIDE),
    (("resize",), dict(cp=_t(I32, [B, 2], [0, 1])), STRIDE),
    (("compact",), dict(mv=_t(I32, [N, 2], [1, 1])), STRIDE),
    (("copy",), dict(k=_t(U8, [NPG, PAGE, HKV, D], data=FAKE + 4)), ALIGN),
    (("copy",), dict(bd=_t(U8, [NPG, HKV, NB, 2, D], data=FAKE + 8)), ALIGN),
    (("copy",), dict(pairs=_t(I32, [N, 2], data=FAKE + 2)), ALIGN),
    (POOL, dict(bt=_t(I32, [B, MP], data=FAKE + 1)), ALIGN),
    (POOL, dict(rc=_t(I32, [NPG], data=FAKE + 2)), ALIGN),
    # workspace
    (("resize",), dict(ws=_t(U8, [128])), WS),
    (("resize",), dict(ws=_t(U8, [1 << 16], data=FAKE + 64)), WS),
])
def test_refusals(lib, names, over, code):
    for name in names:
        a = base()
        a.update(over)
        assert call(lib, name, a) == code, name


@pytest.mark.parametrize("name", NEEDS)
def test_null_tensors_and_pointers(lib, name):
    for k in NEEDS[name]:
        a = base()
        if (name, k) not in (("copy", "sc"), ("copy", "bd")):  # these may be absent
            a[k] = None
            assert call(lib, name, a) == NULL, k
        a = base()
        a[k].data = None
        assert call(lib, name, a) == NULL, k


def test_page_tokens(lib):
    for page in (0, 8, 24, -16, 65552):
        assert call(lib, "resize", base(), page) == UNSUP


def test_nothing_to_do_is_no_error(lib):
    a = base()
    a["pairs"], a["mv"] = _t(I32, [0, 2], data=None), _t(I32, [0, 2], data=None)
    assert call(lib, "copy", a) == 0 and call(lib, "compact", a) == 0
    a.update(bt=_t(I32, [0, MP], data=None), par=_t(I32, [0], data=None), seq=_t(I32, [0, 2], data=None),
             cp=_t(I32, [0, 2], data=None))
    assert call(lib, "fork", a) == 0 and call(lib, "resize", a) == 0


def test_workspace_bytes():
    sums = 128 * 32 * 8  # of the warps of the grid that shares a large pool
    assert vae4.pages_workspace_bytes(1) == sums + 256
    assert vae4.pages_workspace_bytes(1 << 30) == sums + (1 << 32)
    for bad in (0, -1, (1 << 30) + 1):
        with pytest.raises(vae4.Vae4Error):
            vae4.pages_workspace_bytes(bad)


def test_binding_refuses_what_the_library_cannot_see():
    import torch
    c = torch.zeros(2, 16, 1, 64, dtype=torch.uint8)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    for fn in (lambda: vae4.verify_attn_e4m3_copy_pages(c, c, i(1, 2)),
               lambda: vae4.verify_attn_e4m3_fork_pages(i(1, 2), i(4), i(1)),
               lambda: vae4.verify_attn_e4m3_resize_pages(i(1, 2), i(1, 2), i(4), i(1, 2), c.view(-1),
                                                          page_tokens=16),
               lambda: vae4.verify_attn_e4m3_compact_pages(i(1, 2), i(4), i(1, 2))):
        with pytest.raises(ValueError, match="device"):
            fn()
    with pytest.raises(TypeError):  # K and V of different formats
        vae4.verify_attn_e4m3_copy_pages(c.view(torch.float8_e5m2), c.view(torch.float8_e4m3fn), i(1, 2))
    assert vae4.alloc_ref_counts(7, device="cpu").tolist() == [0] * 7
