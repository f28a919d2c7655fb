"""The block-scaled cache's entry points on the host: every refusal comes
before anything is launched.  No compute call is made here."""
import ctypes

import pytest

import fp8_paged_attention_e4m3_gb300 as vae4

FAKE = 0x100000  # never dereferenced: every case below fails validation or has no work


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


U8, I32, F16, F32, BF16 = (vae4.VAE4_U8, vae4.VAE4_I32, vae4.VAE4_F16, vae4.VAE4_F32,
                           vae4.VAE4_BF16)
B, Q, G, HKV, D, PAGE, NB, NPG, MP, K = 2, 8, 6, 2, 128, 96, 2, 40, 16, 5


def base():
    return dict(
        q=_t(F16, [B, Q, G * HKV, D]), x=_t(F16, [B, Q, HKV, D]), y=_t(F16, [B, Q, HKV, D]),
        k=_t(U8, [NPG, PAGE, HKV, D]), v=_t(U8, [NPG, PAGE, HKV, D]),
        bt=_t(I32, [B, MP]), seq=_t(I32, [B, 2]), sc=_t(F32, [NPG, 2, HKV, NB]),
        bd=_t(U8, [NPG, HKV, NB, 2, D]), ids=_t(I32, [B, Q, HKV, K]),
        scores=_t(F32, [B, Q, HKV, 40]), out=_t(F16, [B, Q, G * HKV, D]),
        ws=_t(U8, [1 << 28]))


def call(lib, name, a, opt=None, flags=0, block=48, scale=0.0, sink=0, local=1):
    r = lambda *n: [ctypes.byref(a[k]) if a[k] is not None else None for k in n]  # noqa: E731
    o = ctypes.byref(opt or vae4.Options(0.0, 0, 0, 152, flags, 0))
    if name == "append":
        return lib.verify_attn_e4m3_append(*r("x", "y", "k", "v", "bt", "seq", "sc", "bd"), None,
                                           flags, None)
    if name == "attend":
        return lib.verify_attn_e4m3_block_scaled(*r("q", "k", "v", "bt", "seq", "sc", "out", "ws"),
                                                 None, o)
    if name == "sparse":
        return lib.verify_attn_e4m3_sparse(*r("q", "k", "v", "bt", "seq", "sc", "ids", "out", "ws"),
                                           None, o)
    if name == "scores":
        return lib.verify_attn_e4m3_block_scores(*r("q", "bd", "bt", "seq", "sc", "scores"), block,
                                                 scale, None, flags, None)
    return lib.verify_attn_e4m3_select_blocks(*r("scores", "seq", "ids"), block, sink, local, None,
                                              None)


ALL = ("append", "attend", "sparse", "scores", "select")
NULL, DTYPE, SHAPE, STRIDE, ALIGN, UNSUP, GQA, WS, PART, OPT = (-1, -2, -3, -4, -5, -6, -7, -8,
                                                                -10, -11)


@pytest.mark.parametrize("names,over,code", [
    # types
    (("append",), dict(x=_t(F32, [B, Q, HKV, D])), DTYPE),
    (("append",), dict(y=_t(BF16, [B, Q, HKV, D])), DTYPE),               # K and V differ in type
    (("attend", "sparse", "scores"), dict(q=_t(BF16, [B, Q, G * HKV, D])), DTYPE),
    (("append", "attend", "sparse", "scores"), dict(sc=_t(F16, [NPG, 2, HKV, NB])), DTYPE),
    (("append", "scores"), dict(bd=_t(F16, [NPG, HKV, NB, 2, D])), DTYPE),
    (("sparse", "select"), dict(ids=_t(F32, [B, Q, HKV, K])), DTYPE),
    (("scores", "select"), dict(scores=_t(F16, [B, Q, HKV, 40])), DTYPE),
    (ALL, dict(seq=_t(F32, [B, 2])), DTYPE),
    # shapes
    (("append",), dict(y=_t(F16, [B, Q + 1, HKV, D])), SHAPE),
    (("append",), dict(x=_t(F16, [B, Q, 1, D]), y=_t(F16, [B, Q, 1, D])), SHAPE),
    (("append", "attend", "sparse", "scores"), dict(sc=_t(F32, [HKV, 2])), SHAPE),
    (("append", "attend", "sparse", "scores"), dict(sc=_t(F32, [NPG, 2, 1, NB])), SHAPE),
    (("append", "scores"), dict(bd=_t(U8, [NPG, HKV, NB, D])), SHAPE),
    (("append",), dict(bd=_t(U8, [NPG, HKV, 1, 2, D])), SHAPE),
    (("sparse", "select"), dict(ids=_t(I32, [B, Q, 1, K])), SHAPE),
    (("sparse", "select"), dict(ids=_t(I32, [B, Q, HKV, 0])), SHAPE),
    (("append", "attend", "sparse", "scores"), dict(bt=_t(I32, [B + 1, MP])), SHAPE),
    (ALL, dict(seq=_t(I32, [B, 3])), SHAPE),
    (("scores",), dict(scores=_t(F32, [B, Q, 1, 40])), SHAPE),
    (("append",), dict(bt=_t(I32, [B, 1 << 24])), SHAPE),                 # past 2^30 tokens
    # more KV heads than a segment's record holds
    (("attend",), dict(q=_t(F16, [B, Q, 65536, D]), out=_t(F16, [B, Q, 65536, D]),
                       k=_t(U8, [NPG, PAGE, 65536, D]), v=_t(U8, [NPG, PAGE, 65536, D]),
                       sc=_t(F32, [NPG, 2, 65536, NB])), SHAPE),
    (("scores",), dict(q=_t(F16, [B, Q, 65536, D]), bd=_t(U8, [NPG, 65536, NB, 2, D]),
                       sc=_t(F32, [NPG, 2, 65536, NB]), scores=_t(F32, [B, Q, 65536, 40])), SHAPE),
    # blocks: 24 tokens, 32 tokens of a page of 96 are no multiple / divisor
    (("append", "attend", "sparse"), dict(sc=_t(F32, [NPG, 2, HKV, 4])), UNSUP),
    (("append", "attend", "sparse"), dict(sc=_t(F32, [NPG, 2, HKV, 5])), UNSUP),
    (("append",), dict(x=_t(F16, [B, Q, HKV, 96]), y=_t(F16, [B, Q, HKV, 96])), UNSUP),
    # strides and alignment
    (("append",), dict(x=_t(F16, [B, Q, HKV, D], [Q * HKV * D, HKV * D, D + 4, 1])), STRIDE),
    (("append",), dict(x=_t(F16, [B, Q, HKV, D], data=FAKE + 8)), ALIGN),
    (("append",), dict(k=_t(U8, [NPG, PAGE, HKV, D], [0, HKV * D, D, 1])), STRIDE),  # pages on one another
    (("append",), dict(sc=_t(F32, [NPG, 2, HKV, NB], [0, HKV * NB, NB, 1])), STRIDE),
    (("append",), dict(bd=_t(U8, [NPG, HKV, NB, 2, D], [0, 4 * D, 2 * D, D, 1])), STRIDE),
    (("append", "scores"), dict(bd=_t(U8, [NPG, HKV, NB, 2, D], data=FAKE + 8)), ALIGN),
    (("append", "scores"), dict(bd=_t(U8, [NPG, HKV, NB, 2, D], [2048, 1032, 512, 256, 1])), STRIDE),
    (("sparse", "select"), dict(ids=_t(I32, [B, Q, HKV, K], [Q * HKV * K, HKV * K, K, 2])), STRIDE),
    (("select",), dict(ids=_t(I32, [B, Q, HKV, K], [Q * HKV * K, HKV * K, 0, 1])), STRIDE),
    (("scores",), dict(scores=_t(F32, [B, Q, HKV, 40], [0, HKV * 40, 40, 1])), STRIDE),
    (("scores", "select"), dict(scores=_t(F32, [B, Q, HKV, 40], data=FAKE + 2)), ALIGN),
    # heads, workspace, rows
    (("attend", "sparse", "scores"), dict(q=_t(F16, [B, Q, 7, D]), out=_t(F16, [B, Q, 7, D])), GQA),
    (("attend", "sparse"), dict(ws=_t(U8, [1000])), WS),
    (("attend", "sparse", "scores"), dict(q=_t(F16, [B, Q, 32, D]), out=_t(F16, [B, Q, 32, D])), UNSUP),
])
def test_refusals(lib, names, over, code):
    for name in names:
        a = base()
        a.update(over)
        assert call(lib, name, a) == code, name


@pytest.mark.parametrize("name,needs", [
    ("append", ("x", "y", "k", "v", "bt", "seq", "sc")),
    ("attend", ("q", "k", "v", "bt", "seq", "sc", "out", "ws")),
    ("sparse", ("q", "k", "v", "bt", "seq", "sc", "ids", "out", "ws")),
    ("scores", ("q", "bd", "bt", "seq", "sc", "scores")),
    ("select", ("scores", "seq", "ids")),
])
def test_null_tensors_and_pointers(lib, name, needs):
    for k in needs:
        a = base()
        a[k] = None
        assert call(lib, name, a) == NULL, k
        a = base()
        a[k].data = None
        assert call(lib, name, a) == NULL, k


def test_options(lib):
    o = lambda **kw: vae4.Options(kw.get("s", 0.0), kw.get("T", 0), kw.get("cap", 0), 152,  # noqa: E731
                                  kw.get("flags", 0), kw.get("hilo", 0))
    for name in ("attend", "sparse"):
        assert call(lib, name, base(), o(flags=vae4.FLAG_WARP_MMA)) == UNSUP
        assert call(lib, name, base(), o(hilo=1)) == UNSUP
        assert call(lib, name, base(), o(hilo=2)) == OPT
        assert call(lib, name, base(), o(flags=16)) == OPT
        assert call(lib, name, base(), o(s=-1.0)) == OPT
        assert call(lib, name, base(), o(cap=MP * PAGE + 1)) == SHAPE
    for name in ("attend", "sparse"):  # the keys are divided on the device
        for T in (24, 64):
            assert call(lib, name, base(), o(T=T)) == PART
    for name in ("append", "scores"):
        assert call(lib, name, base(), flags=vae4.FLAG_WARP_MMA) == OPT
    assert call(lib, "scores", base(), scale=-1.0) == OPT
    assert call(lib, "scores", base(), scale=float("nan")) == OPT
    for block in (0, 8, 24, -16, 65536):  # 2 blocks of a page: the page would pass 65536
        assert call(lib, "scores", base(), block=block) == UNSUP
    assert call(lib, "select", base(), block=40) == UNSUP
    assert call(lib, "select", base(), sink=-1) == OPT
    assert call(lib, "select", base(), sink=3, local=3) == OPT  # more than k = 5
    # the most blocks a visit list can hold
    a = base()
    a["sc"], a["k"], a["v"] = (_t(F32, [NPG, 2, HKV, 1]), _t(U8, [NPG, 16, HKV, D]),
                               _t(U8, [NPG, 16, HKV, D]))
    a["bt"], a["ws"] = _t(I32, [B, 98305]), _t(U8, [1000])
    assert call(lib, "sparse", a) == UNSUP
    assert call(lib, "sparse", a, o(cap=98304 * 16)) == WS  # within it


def test_empty_batch_is_no_error(lib):
    a = base()
    for k, shape in dict(q=[0, Q, G * HKV, D], x=[0, Q, HKV, D], y=[0, Q, HKV, D], bt=[0, MP],
                         seq=[0, 2], ids=[0, Q, HKV, K], scores=[0, Q, HKV, 40],
                         out=[0, Q, G * HKV, D]).items():
        a[k] = _t(a[k].dtype, shape, data=None)
    for name in ALL:
        assert call(lib, name, a) == 0, name


def test_workspace_bytes():
    """Status, partial states of two units per SM (fewer SMs if there are fewer
    64-key pieces), the units' table; sparse: stream records and lists."""
    al = lambda x: (x + 255) // 256 * 256  # noqa: E731

    def dense(streams, n_rg, N, D, pieces):
        ctas = min(152, streams * n_rg * pieces)
        o = al(al(256 + 2 * ctas * N * 8) + 2 * ctas * N * D * 4)
        return o + streams * n_rg * 8

    bs = vae4.block_scaled_workspace_bytes
    assert bs(2, 12, 2, 8, D, 1536, 152) == dense(4, 1, 48, D, 24)    # 48 rows
    assert bs(1, 6, 1, 16, 256, 262144, 152) == dense(1, 2, 48, 256, 4096)  # two row groups
    assert bs(1, 2, 1, 1, 64, 100, 152) == dense(1, 1, 16, 64, 2)     # two pieces
    # beyond 4096 CTAs the combine would not hold a unit's parts
    assert bs(1, 2, 1, 1, 64, 1 << 20, 4096) == bs(1, 2, 1, 1, 64, 1 << 20, 10000)
    # 2 sequences x 2 KV heads, 5 blocks of 48 tokens for each of 8 queries
    entries = min(-(-1536 // 48), 8 * 5)
    n = al(al(dense(4, 1, 48, D, 24)) + 4 * 16) + 4 * entries * 32
    assert vae4.sparse_workspace_bytes(2, 12, 2, 8, D, 1536, 48, 5, 152) == n
    for bad in ((1, 7, 2, 8, D, 1536), (1, 12, 2, 8, 96, 1536), (1, 12, 2, 17, D, 1536),
                (1, 12, 2, 8, D, 0), (0, 12, 2, 8, D, 1536), (1, 32, 1, 4, D, 1536)):
        with pytest.raises(vae4.Vae4Error):
            bs(*bad, 152)
        with pytest.raises(vae4.Vae4Error):
            vae4.sparse_workspace_bytes(*bad, 48, 5, 152)
    for bad in ((1, 12, 2, 8, D, 1536, 40, 5), (1, 12, 2, 8, D, 1536, 48, 0),
                (1, 12, 2, 8, D, 16 * 98305, 16, 5)):
        with pytest.raises(vae4.Vae4Error):
            vae4.sparse_workspace_bytes(*bad, 152)


def test_binding_refuses_what_the_library_cannot_see():
    """CPU tensors (whose pointers mean nothing on the device) are refused by
    the binding; the allocation helpers check the block."""
    import torch
    x = torch.zeros(1, 1, 1, 64, dtype=torch.float16)
    c = torch.zeros(2, 16, 1, 64, dtype=torch.uint8)
    bt, seq = torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, 2, dtype=torch.int32)
    sc, ids = torch.ones(2, 2, 1, 1), torch.zeros(1, 1, 1, 1, dtype=torch.int32)
    bd, scores = torch.zeros(2, 1, 1, 2, 64, dtype=torch.uint8), torch.zeros(1, 1, 1, 1)
    ws = torch.zeros(1024, dtype=torch.uint8)
    for fn in (lambda: vae4.verify_attn_e4m3_append(x, x, c, c, bt, seq, sc),
               lambda: vae4.verify_attn_e4m3_block_scaled(x, c, c, bt, seq, sc, x, ws),
               lambda: vae4.verify_attn_e4m3_sparse(x, c, c, bt, seq, sc, ids, x, ws),
               lambda: vae4.verify_attn_e4m3_block_scores(x, bd, bt, seq, sc, scores, block_tokens=16),
               lambda: vae4.verify_attn_e4m3_select_blocks(scores, seq, ids, block_tokens=16)):
        with pytest.raises(ValueError, match="device"):
            fn()
    with pytest.raises(ValueError):
        vae4.alloc_block_scales(2, 1, 96, 40, device="cpu")
    with pytest.raises(ValueError):
        vae4.alloc_k_bounds(2, 1, 96, 24, 64, device="cpu")
    assert vae4.alloc_block_scales(2, 3, 96, 48, device="cpu").shape == (2, 2, 3, 2)
    assert vae4.alloc_k_bounds(2, 3, 96, 48, 64, device="cpu").shape == (2, 3, 2, 2, 64)
    k, v = vae4.cache_views(torch.arange(2 * 2 * 3 * 16 * 64).view(2, 2, 3, 16, 64))
    assert k.shape == v.shape == (2, 16, 3, 64) and int(v[0, 0, 0, 0]) == 3 * 16 * 64
