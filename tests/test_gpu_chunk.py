"""Chunk attention on the GPU against its definition in 64 bits (torch on the
device's FP64 units, sharing no code with the kernels).

Tolerance, derived from the arithmetic: a weight w_t = e^(z_t - max z) s_V enters
the value product rounded to FP16, so off by at most 2^-11 of itself, or, below
2^-14 of the row's largest, W, by at most 2^-25 W; the FP32 score of a key is off
by far less than 2^-11 in log2 units at these sizes, which the factor 2 in 2^-10
covers together with the FP32 sums; out is rounded once, by at most half a step
(2^-11 of it in FP16, 2^-8 in BF16; below FP16's normal range by 2^-25).  With
l = sum e^(z_t - max z) and A = sum e^(z_t - max z) |V_t| / l:
    |got - out| <= half |out| + 2^-10 (A + |out|) + 2^-25 W sum |dec(V_t)| / l + 2^-24
"""
import math

import pytest
import torch

import fp8_paged_attention_e4m3_gb300 as vae4
from test_gpu_blocks import FMT, Cache, dev

pytestmark = pytest.mark.gpu

KIND = {"f16": (torch.float16, 2.0 ** -11), "bf16": (torch.bfloat16, 2.0 ** -8)}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    vae4.load()


def per_head(c, seed=0):
    """The cache's codes with one scale per KV head, and what they stand for."""
    g = torch.Generator().manual_seed(seed)
    c.head = torch.exp2(torch.randint(-9, -5, (c.Hkv, 2), generator=g).float()) * (1 + torch.rand(c.Hkv, 2, generator=g))
    return c


def codes(c, w, b):
    """(dec, scale) of the L tokens of sequence b, [L][Hkv][D] and [L][Hkv], FP64."""
    L = c.lens[b][0]
    pg = c.table[b, :-(-L // c.page)].long()
    x = c.codes[w][pg].view(FMT[c.fmt][0]).double().flatten(0, 1)[:L].cuda()
    if hasattr(c, "head"):
        s = c.head[:, w].double().expand(L, -1)
    else:
        s = c.scales[pg, w].double().repeat_interleave(c.blk, 2).transpose(1, 2).flatten(0, 1)[:L]
    return x, s.cuda()


def reference(c, q, scale=0.0):
    """(out, bound); rows past a sequence's queries are NaN in out."""
    B, Q, Hq, D = q.shape
    G, half = Hq // c.Hkv, KIND["bf16" if q.dtype == torch.bfloat16 else "f16"][1]
    sm = scale or 1 / math.sqrt(D)
    out = torch.full((B, Q, Hq, D), float("nan"), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    for b, (L, n) in enumerate(c.lens):
        if L == 0:
            out[b, :n] = 0
            continue
        (K, sk), (V, sv) = codes(c, 0, b), codes(c, 1, b)
        for i0 in range(0, n, 512):
            x = q[b, i0:min(i0 + 512, n)].cuda().double()
            m = x.shape[0]
            i = L - n + i0 + torch.arange(m, device="cuda")
            hide = torch.arange(L, device="cuda") > i[:, None]
            for h in range(c.Hkv):
                z = torch.einsum("igd,td->igt", x[:, h * G:(h + 1) * G], K[:, h] * sk[:, h, None]) * sm
                z.masked_fill_(hide[:, None], float("-inf"))
                e = torch.exp(z - z.amax(-1, keepdim=True))
                l = e.sum(-1, keepdim=True)
                w = e * sv[:, h] / l
                o, a = w @ V[:, h], w @ V[:, h].abs()
                seen = (~hide).double() @ V[:, h].abs()
                W = w.amax(-1, keepdim=True)
                out[b, i0:i0 + m, h * G:(h + 1) * G] = o
                tol[b, i0:i0 + m, h * G:(h + 1) * G] = (half * o.abs() + 2.0 ** -10 * (a + o.abs()) +
                                                        2.0 ** -25 * W * seen[:, None] + 2.0 ** -24)
    return out, tol


def queries(c, Q, G, kind="f16", seed=1):
    """Queries of heads of different sharpness; the padding slots hold NaN."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(len(c.lens), Q, G * c.Hkv, c.D, generator=g)
    q *= torch.exp2(torch.rand(1, 1, G * c.Hkv, 1, generator=g) * 2 - 1)
    q = q.to(KIND[kind][0])
    for b, (_, n) in enumerate(c.lens):
        q[b, max(n, 0):] = float("nan")
    return q


MARK = 7.0  # what out holds before the call


def attend(c, q, layout="tokens", out=None, **kw):
    B, Q, Hq, D = q.shape
    cap = kw.pop("max_seq_len", 0)
    k, v = c.device(layout)
    qd = q if q.is_cuda else q.cuda()
    bt, seq, sc = dev(c.table, c.seq, c.head if hasattr(c, "head") else c.scales)
    if out is None:
        out = torch.full(q.shape, MARK, dtype=q.dtype, device="cuda")
    top = cap or c.table.shape[1] * c.page
    n = vae4.chunk_workspace_bytes(B, Hq, c.Hkv, Q, D, top, kw.get("num_sms", 0))
    ws = torch.zeros(n + 256, dtype=torch.uint8, device="cuda")
    ws[n:] = 0x5A  # nothing past the workspace is written
    flags = kw.pop("flags", 0) | FMT[c.fmt][2]
    vae4.verify_attn_e4m3_chunk(qd, k, v, bt, seq, sc, out, ws[:n], max_seq_len=cap, flags=flags, **kw)
    torch.cuda.synchronize()
    assert bool((ws[n:] == 0x5A).all())
    return out, vae4.read_status(ws[:n])


def check(got, ref, tol):
    """Rows of queries within the bound, the others as they were."""
    pad = ref.isnan()
    assert bool((got[pad] == MARK).all())
    far = ((got.double() - ref).abs() - tol)[~pad]
    assert bool((far <= 0).all()), f"{far.max().item()} past the bound"  # (a NaN is not <= 0)


CASES = [
    # lens, Q, G, Hkv, D, page, block, format, layout, type, scales
    ([(1, 1)], 1, 1, 1, 64, 16, 16, "e4m3", "tokens", "f16", "block"),
    ([(2, 2)], 2, 1, 1, 128, 16, 16, "e4m3", "pool", "bf16", "head"),
    ([(17, 17)], 17, 3, 1, 256, 16, 16, "e4m3", "tokens", "f16", "block"),
    ([(128, 128)], 128, 1, 1, 128, 16, 16, "e4m3", "tokens", "f16", "block"),
    ([(129, 129)], 129, 2, 1, 128, 16, 16, "e4m3", "tokens", "bf16", "block"),
    ([(257, 256)], 256, 1, 1, 64, 64, 32, "e4m3", "pool", "f16", "head"),
    ([(1000, 1000)], 1000, 2, 1, 128, 48, 16, "e4m3", "tokens", "f16", "block"),
    ([(1000, 1000)], 1000, 2, 2, 64, 48, 48, "e5m2", "tokens", "bf16", "block"),
    ([(777, 500)], 500, 3, 1, 256, 48, 48, "e4m3", "pool", "bf16", "block"),
    ([(2049, 2049)], 2049, 1, 1, 128, 96, 32, "e4m3", "tokens", "bf16", "head"),
    ([(700, 257), (129, 1), (0, 0), (128, 128), (1000, 16), (16, 0), (300, 299)], 300, 6, 2, 128, 32, 16, "e4m3",
     "tokens", "f16", "block"),
    ([(700, 257), (129, 1), (0, 5), (128, 128), (1000, 16), (300, 299)], 300, 5, 3, 64, 64, 64, "e5m2", "pool", "f16",
     "head"),
    ([(400, 57), (129, 1), (128, 128), (1000, 16), (300, 299)], 300, 6, 1, 256, 16, 16, "e4m3", "padded", "f16",
     "block"),
    ([(1500, 40), (300, 8)], 41, 4, 2, 128, 32, 16, "e5m2", "padded", "bf16", "block"),
    ([(20000, 33)], 33, 6, 1, 256, 16, 16, "e4m3", "tokens", "f16", "block"),
    ([(30011, 19)], 19, 16, 1, 128, 848, 848, "e4m3", "pool", "bf16", "block"),
    ([(9000, 3), (40, 40)], 40, 1, 8, 64, 128, 16, "e4m3", "tokens", "f16", "block"),
    ([(3000, 1200)], 1200, 16, 1, 64, 64, 64, "e4m3", "tokens", "f16", "head"),
    ([(5, 1)] * 300, 1, 2, 2, 64, 16, 16, "e4m3", "tokens", "f16", "block"),
    ([(1 + b, 1 + b % (b + 1)) for b in range(70)], 71, 4, 3, 128, 32, 32, "e4m3", "tokens", "bf16", "head"),
    ([(1 + b % 200, 1) for b in range(2500)], 1, 1, 1, 128, 16, 16, "e4m3", "tokens", "f16", "block"),
    ([(130, 129)] * 33, 129, 8, 2, 256, 64, 64, "e4m3", "pool", "bf16", "block"),
    ([(64, 64)], 64, 96, 1, 128, 64, 64, "e4m3", "tokens", "f16", "block"),  # 96 heads on one
]


@pytest.mark.parametrize("lens,Q,G,Hkv,D,page,blk,fmt,layout,kind,scales", CASES,
                         ids=[f"{len(c[0])}x{c[3]}-q{c[1]}x{c[2]}-{c[4]}-{'-'.join(map(str, c[5:]))}" for c in CASES])
def test_the_definition(lens, Q, G, Hkv, D, page, blk, fmt, layout, kind, scales):
    c = Cache(lens, Hkv, D, page, blk, fmt, seed=len(lens) + D)
    if scales == "head":
        per_head(c, D)
    q = queries(c, Q, G, kind)
    got, status = attend(c, q, layout)
    assert status == 0
    check(got, *reference(c, q))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_every_code(D, fmt, kind):
    """Keys whose channel d holds every finite code, queries of one channel each:
    the scores, and with them the weights, are those of the codes."""
    c = Cache([(256, D)], 1, D, 256, 256, fmt, seed=1)
    c.scales[:] = 2.0 ** -6 if fmt == "e4m3" else 2.0 ** -13
    pg = int(c.table[0, 0])
    code = torch.arange(256, dtype=torch.uint8)
    code[~torch.isfinite(code.view(FMT[fmt][0]).float())] = 0
    c.codes[0][pg] = torch.stack([code.roll(d) for d in range(D)], -1)[:, None, :]
    q = torch.zeros(1, D, 1, D, dtype=KIND[kind][0])
    q[0, range(D), 0, range(D)] = 8.0
    got, status = attend(c, q, softmax_scale=0.125)
    assert status == 0
    check(got, *reference(c, q, 0.125))


@pytest.mark.parametrize("sms", [1, 2, 7, 152, 400])
def test_other_numbers_of_sms(sms):
    """One CTA walks all, units are shared by two and by many; twice the same bits."""
    c = Cache([(1000, 300), (130, 1), (64, 2), (4000, 33), (0, 0), (700, 200)], 2, 128, 32, 16, seed=12)
    q = queries(c, 300, 3)
    got, status = attend(c, q, num_sms=sms)
    assert status == 0
    check(got, *reference(c, q))
    assert torch.equal(got, attend(c, q, num_sms=sms)[0])


@pytest.mark.parametrize("D,G,n", [(128, 2, 1300), (256, 3, 400), (64, 1, 2000)])
def test_every_row_of_a_long_chunk(D, G, n):
    """Long chunks behind a context, shared by all SMs at odd places."""
    c = Cache([(n + 1777, n)], 1, D, 64, 64, seed=D)
    q = queries(c, n, G, "bf16")
    got, status = attend(c, q)
    assert status == 0
    check(got, *reference(c, q))


def test_scales_far_apart():
    """Blocks whose V scales differ by up to 2^40."""
    c = Cache([(640, 200)], 2, 128, 64, 16, seed=5)
    g = torch.Generator().manual_seed(9)
    e = torch.randint(-20, 21, c.scales[:, 1].shape, generator=g)
    e[int(c.table[0, 0])], e[int(c.table[0, 1])] = -20, 20
    c.scales[:, 1] = torch.where(c.scales[:, 1].isnan(), c.scales[:, 1], torch.exp2(e.float() - 18))
    q = queries(c, 200, 3)
    ref, tol = reference(c, q)
    assert ref.abs().max() < 6e4
    got, status = attend(c, q)
    assert status == 0
    check(got, ref, tol)


def test_scores_that_grow_along_the_context():
    """Later keys beat the earlier ones by far, so every row's reference is raised
    many times, the accumulator with it."""
    c = Cache([(1500, 260)], 1, 128, 64, 64, seed=6)
    c.scales[:, 0] *= 8
    for j in range(24):
        pg = int(c.table[0, j])
        c.scales[pg, 0] *= 1 + 0.4 * j
    q = queries(c, 260, 2)
    got, status = attend(c, q)
    assert status == 0
    ref, tol = reference(c, q)
    # scores of up to some hundreds: 2^-22 of them beside the weights' own rounding
    z = 128 ** 0.5 * 3 * float(c.scales[c.table[0, :24].long(), 0].max()) * 448
    check(got, ref, tol + ref.abs().max() * z * 2.0 ** -21)


def test_lengths_without_q_softmax_scale_and_capacity():
    c = Cache([(100, 33), (40, 33)], 1, 64, 32, 16, seed=3)
    q = queries(c, 33, 5)
    ref = reference(c, q, 0.31)
    c.seq = torch.tensor([100, 40], dtype=torch.int32)  # q = Qmax for all
    got, status = attend(c, q, softmax_scale=0.31, max_seq_len=100)
    assert status == 0
    check(got, *ref)


def test_queries_without_numbers():
    """NaN, infinite and zero queries: rows of their own, the others not concerned."""
    c = Cache([(400, 140)], 1, 128, 32, 16, seed=8)
    q = queries(c, 140, 2)
    want, _ = attend(c, q)
    q[0, 3, 0, 5], q[0, 77, 1, 0] = float("nan"), float("inf")
    q[0, 130] = 0
    ref, tol = reference(c, q)
    got, status = attend(c, q)
    assert status == 0
    odd = torch.zeros(140, 2, dtype=torch.bool)
    odd[3, 0] = odd[77, 1] = True
    assert bool(got[0][odd].isnan().all())
    same = ~odd
    same[130] = False
    assert torch.equal(got[0][same], want[0][same])
    far = ((got.double() - ref).abs() - tol)[0, 130]
    assert bool((far <= 0).all())


def test_scores_of_minus_infinity():
    """All scores -infinity: zeros; some: the others decide."""
    c = Cache([(200, 30)], 1, 64, 32, 16, seed=8)
    pages = c.table[0, :7].long()
    c.codes[0][pages] = (c.codes[0][pages] & 0x7F).clamp(8, 0x70)  # positive
    q = torch.ones(1, 30, 1, 64, dtype=torch.float16)
    q[0, 4] = float("-inf")
    got, status = attend(c, q)
    assert status == 0 and not got[0, 4].any() and not got.isnan().any()


def test_invalid_pages_scales_and_lengths():
    """A row that sees an invalid page or block is zero, the rows before it are not
    concerned; nor are other heads."""
    lens = [(400, 300), (300, 150), (250, 2), (90, 90), (50, 5), (30, 31)]
    for D, G in ((128, 2), (256, 1)):
        c = Cache(lens, 2, D, 32, 16, seed=4)
        q = queries(c, 300, G)
        ref, tol = reference(c, q)
        c.table[0, 8] = c.n_pages             # tokens 256 .. 287 of sequence 0
        pg = int(c.table[1, 7])
        c.scales[pg, 1, 1, 1] = float("inf")  # sequence 1, KV head 1: tokens 240 .. 255
        c.table[3, 0] = -1
        c.seq[2, 0] = 100000                  # longer than the table
        got, status = attend(c, q)
        assert status == (vae4.STATUS_BAD_BLOCK | vae4.STATUS_BAD_SCALE | vae4.STATUS_BAD_LENGTH |
                          vae4.STATUS_BAD_QLEN)
        zero = torch.zeros(ref.shape, dtype=torch.bool)
        zero[0, 256 - 100:300] = True
        zero[1, 240 - 150:150, G:] = True
        zero[2, :2] = zero[3, :90] = zero[5, :31] = True
        ref[zero] = tol[zero] = 0
        check(got, ref, tol)
    for bad in (0.0, -1.0, float("nan"), 2.0 ** 41, 2.0 ** -41):
        c = per_head(Cache([(90, 80)], 2, 64, 32, 16, seed=4))
        c.head[1, 0] = bad
        got, status = attend(c, queries(c, 80, 2))
        assert status == vae4.STATUS_BAD_SCALE and not got[:, :, 2:].any() and bool((got[:, :, :2] != 0).any())


def test_strided_queries_and_outputs():
    """Heads outermost with space between, a query used by two sequences."""
    c = Cache([(300, 130), (200, 130)], 2, 128, 32, 16, seed=9)
    q1 = queries(c, 130, 3)[:1]
    q = q1.expand(2, -1, -1, -1).cuda()  # stride 0
    wide = torch.full((6, 2, 131, 144), MARK, dtype=torch.float16, device="cuda")
    out = wide[:, :, :130, 8:136].permute(1, 2, 0, 3)
    got, status = attend(c, q, out=out)
    assert status == 0
    check(got, *reference(c, q))
    rest = wide.clone()
    rest[:, :, :130, 8:136] = MARK
    assert bool((rest == MARK).all())


def test_offsets_past_32_bits():
    """Pages whose bytes lie past 2^32, in K and in V."""
    n_pages, page, H, D = 36, 65536, 8, 256
    lens = [(200, 150)]
    c = Cache(lens, H, D, 208, 208, seed=2)
    k, v = [torch.zeros(n_pages, page, H, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    pg = int(c.table[0, 0])
    k[35, :208], v[35, :208] = c.codes[0][pg].cuda(), c.codes[1][pg].cuda()
    sc = torch.ones(n_pages, 2, H, 1, device="cuda")
    sc[35] = c.scales[pg].cuda()
    q = queries(c, 150, 1)
    out = torch.full(q.shape, MARK, dtype=q.dtype, device="cuda")
    ws = vae4.alloc_chunk_workspace(1, H, H, 150, D, page)
    bt = torch.full((1, 1), 35, dtype=torch.int32, device="cuda")
    vae4.verify_attn_e4m3_chunk(q.cuda(), k, v, bt, c.seq.cuda(), sc, out, ws)
    assert vae4.read_status(ws) == 0
    check(out, *reference(c, q))


def test_waits_that_run_out_mark_the_rows():
    """Every pipeline wait gives up at once: the call reports the timeout and writes
    zero rows, and the workspace serves the next call."""
    for D in (64, 128, 256):
        c = Cache([(3000, 40), (100, 100), (50, 2), (9000, 5)], 2, D, 32, 16, seed=13)
        q = queries(c, 100, 3)
        ref, tol = reference(c, q)
        k, v = c.device()
        qd, bt, seq, sc = dev(q, c.table, c.seq, c.scales)
        ws = vae4.alloc_chunk_workspace(4, 6, 2, 100, D, c.table.shape[1] * c.page)
        for flags in (vae4.FLAG_TEST_SHORT_WAITS, 0):
            out = torch.full_like(qd, MARK)
            vae4.verify_attn_e4m3_chunk(qd, k, v, bt, seq, sc, out, ws, flags=flags)
            torch.cuda.synchronize()
            assert vae4.read_status(ws) == (vae4.STATUS_TIMEOUT if flags else 0)
            vae4.clear_status(ws)
            check(out, torch.where(ref.isnan(), ref, 0.0) if flags else ref, tol * (not flags))


def test_beside_block_scaled_attention():
    """Up to 16 queries: both calls within their bounds of the same definition."""
    c = Cache([(3000, 8), (100, 5), (7, 7)], 2, 128, 32, 16, seed=13)
    q = queries(c, 8, 3)
    ref, tol = reference(c, q)
    got, _ = attend(c, q)
    check(got, ref, tol)
    k, v = c.device()
    qd, bt, seq, sc = dev(q, c.table, c.seq, c.scales)
    out, ws = torch.empty_like(qd), vae4.alloc_workspace(3, 6, 2, 8, 128, c.table.shape[1] * c.page)
    vae4.verify_attn_e4m3_block_scaled(qd, k, v, bt, seq, sc, out, ws)
    live = ~ref.isnan()
    assert bool(((out.double() - got.double()).abs() <= 2 * tol)[live].all())


def test_two_streams_and_a_captured_graph():
    """Calls at once on two streams with workspaces of their own; a captured call
    replayed with other lengths."""
    c = Cache([(6000, 200), (900, 3), (3100, 100)], 2, 128, 32, 16, seed=15)
    q = queries(c, 200, 4)
    k, v = c.device()
    bt, seq, sc = dev(c.table, c.seq, c.scales)
    qd = q.cuda()
    cap = c.table.shape[1] * c.page
    want, _ = attend(c, q)
    ws = [vae4.alloc_chunk_workspace(3, 8, 2, 200, 128, cap) for _ in range(2)]
    outs = torch.full((2, 8) + q.shape, MARK, dtype=q.dtype, device="cuda")
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for n in range(8):
        for x in range(2):
            vae4.verify_attn_e4m3_chunk(qd, k, v, bt, seq, sc, outs[x, n], ws[x], stream=streams[x])
    torch.cuda.synchronize()
    assert bool((outs == want).all())
    graph, out = torch.cuda.CUDAGraph(), torch.full_like(qd, MARK)
    with torch.cuda.graph(graph):
        vae4.verify_attn_e4m3_chunk(qd, k, v, bt, seq, sc, out, ws[0])
    for lens in ([(6000, 200), (900, 3), (3100, 100)], [(10, 10), (0, 0), (2000, 200)], [(1, 1), (900, 3), (5000, 0)]):
        c.lens = [(min(L, 3100) if b else L, n) for b, (L, n) in enumerate(lens)]
        c.seq = torch.tensor(c.lens, dtype=torch.int32)
        seq.copy_(c.seq)
        qd.copy_(queries(c, 200, 4))
        out.fill_(MARK)
        graph.replay()
        torch.cuda.synchronize()
        check(out, *reference(c, qd.cpu()))
    assert all(vae4.read_status(w) == 0 for w in ws)


def test_a_prompt_in_chunks_shared_and_continued():
    """resize, append and chunk attention, then a fork, copies of its last page and
    single tokens: each step against its definition over the cache as it is."""
    B, cols, page, blk, H, G, D, n_pages = 3, 20, 32, 16, 2, 3, 128, 50
    g = torch.Generator().manual_seed(3)
    table = torch.full((B, cols), -1, dtype=torch.int32, device="cuda")
    counts, pws = vae4.alloc_ref_counts(n_pages), vae4.alloc_pages_workspace(n_pages)
    copies = torch.empty((B, 2), dtype=torch.int32, device="cuda")
    kv = torch.full((n_pages, 2, H, page, D), 0x7F, dtype=torch.uint8, device="cuda")
    k, v = vae4.cache_views(kv)
    scales = vae4.alloc_block_scales(n_pages, H, page, blk)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = vae4.alloc_chunk_workspace(B, H * G, H, 150, D, cols * page)
    lens = [(0, 0)] * B

    class Now:  # the cache as it is
        Hkv, fmt = H, "e4m3"

    def step(q):
        nonlocal lens
        lens = [(L + n, n) for (L, _), n in zip(lens, q)]
        seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
        vae4.verify_attn_e4m3_resize_pages(table, seq, counts, copies, pws, page_tokens=page, status=st)
        vae4.verify_attn_e4m3_copy_pages(k, v, copies, block_scales=scales, status=st)
        new = [torch.randn(B, max(q), H, D, generator=g).bfloat16().cuda() for _ in range(2)]
        vae4.verify_attn_e4m3_append(*new, k, v, table, seq, scales, status=st)
        x = torch.randn(B, max(q), H * G, D, generator=g).bfloat16().cuda()
        out = torch.full_like(x, MARK)
        vae4.verify_attn_e4m3_chunk(x, k, v, table, seq, scales, out, ws)
        c = Now()
        c.lens, c.page, c.blk, c.table, c.scales, c.codes = lens, page, blk, table.cpu(), scales.cpu(), [k.cpu(), v.cpu()]
        check(out, *reference(c, x))

    for q in ([150, 7, 0], [101, 0, 0], [1, 50, 0], [77, 1, 0]):
        step(q)
    vae4.verify_attn_e4m3_fork_pages(table, counts, torch.tensor([0, 0, 1], dtype=torch.int32, device="cuda"), status=st)
    lens = [lens[0], lens[0], lens[1]]
    for q in ([1, 1, 1], [8, 3, 150], [1, 1, 1]):
        step(q)
    assert int(st) == 0 and vae4.read_status(ws) == 0
    assert bool((copies == -1).all())  # by now every row's last page is its own
    lens = [(0, 0)] * B
    step([0, 0, 5])
    assert int((counts > 0).sum()) == 1


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("sms", [0, 8])
def test_repeated_calls_give_the_same_bits(D, sms):
    """100 calls behind one another, units shared by few and by many CTAs."""
    c = Cache([(9000, 33), (700, 300)], 1, D, 16, 16, seed=D)
    q = queries(c, 300, 6)
    k, v = c.device()
    qd, bt, seq, sc = dev(q, c.table, c.seq, c.scales)
    ws = torch.zeros(vae4.chunk_workspace_bytes(2, 6, 1, 300, D, c.table.shape[1] * 16, sms), dtype=torch.uint8,
                     device="cuda")
    outs = torch.full((100,) + q.shape, MARK, dtype=q.dtype, device="cuda")
    for out in outs:
        vae4.verify_attn_e4m3_chunk(qd, k, v, bt, seq, sc, out, ws, num_sms=sms)
    assert bool((outs == outs[0]).all()) and vae4.read_status(ws) == 0
    check(outs[0], *reference(c, q))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("sms", [2, 12])
def test_units_of_every_number_of_tiles_in_turn(D, sms):
    """Few rows and many, one tile of keys and several, one unit after another on the
    same SMs: two accumulators that take the tiles in turn, or one alone."""
    lens = []
    for n in range(1, 12):
        lens += [(128 * n - 5, 1), (3, 1), (128 * n + 131, 130), (100, 40), (64, 64), (700, 1)]
    c = Cache(lens, 2, D, 32, 16, seed=D)
    q = queries(c, 130, 3)
    got, status = attend(c, q, num_sms=sms)
    assert status == 0
    check(got, *reference(c, q))
    assert torch.equal(got, attend(c, q, num_sms=sms)[0])
