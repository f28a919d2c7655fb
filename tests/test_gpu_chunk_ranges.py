"""Chunk attention on the GPU at the ends of its number ranges, against its definition in
64 bits; caches, definition and the derivation of the bound are those of test_gpu_chunk."""
import math

import pytest
import torch

import fp8_paged_attention_e4m3_gb300 as vae4
from test_gpu_blocks import Cache
from test_gpu_chunk import KIND, attend, check, codes, queries, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    vae4.load()


# lens of which rows lie in masked tiles, whole and alone, in one unit and in several
LENS = [(300, 300), (900, 40), (17, 1)]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("power,scale_k", [(-100, -40), (-120, -40), (-120, -30), (-133, -40), (-93, -40), (-110, 40)])
def test_small_queries_and_small_scales(D, power, scale_k):
    """BF16 queries of 2^power beside K scales of 2^scale_k: what a score is multiplied with
    may be too small for 32 bits.  All scores are next to zero, hidden keys stay hidden."""
    c = Cache(LENS, 2, D, 32, 16, seed=D)
    c.scales[:, 0] = torch.where(c.scales[:, 0].isnan(), c.scales[:, 0], 2.0 ** scale_k)
    q = (queries(c, 300, 2, "f16").double() * 2.0 ** power).bfloat16()  # (NaN in the padding still)
    q[0, 5] = 0
    got, status = attend(c, q)
    assert status == 0
    check(got, *reference(c, q))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("scale", [1e-30, 1e-36, 1e-38, 1e-44])
def test_small_softmax_scales(D, kind, scale):
    c = Cache(LENS, 2, D, 32, 16, seed=D)
    q = queries(c, 300, 2, kind)
    got, status = attend(c, q, softmax_scale=scale)
    assert status == 0
    check(got, *reference(c, q, scale))


FACTORS = [("bf16", 100, 0.0), ("bf16", 120, 0.0), ("f16", 3, 1e30), ("bf16", 60, 1e25)]  # queries, softmax_scale


def past_32_bits(D, lens, signs, kind, power, scale):
    """Queries of one large value; keys of zeros, every other one of the sequence's sign,
    so that a score is 0 or past 2^128."""
    c = Cache(lens, 1, D, 32, 16, seed=D)
    for b, sign in enumerate(signs):
        pg = c.table[b, :-(-lens[b][0] // 32)].long()
        k = c.codes[0][pg]
        k[:, 0::2] = 0
        k[:, 1::2] = (k[:, 1::2] & 0x7F).clamp(0x38, 0x70) | sign
        c.codes[0][pg] = k
    c.scales[:, 0] = torch.where(c.scales[:, 0].isnan(), c.scales[:, 0], 2.0 ** 40)
    q = torch.full((len(lens), 300, 2, D), 2.0 ** power).to(KIND[kind][0])
    for b, (_, n) in enumerate(lens):
        q[b, n:] = float("nan")
    assert math.log2(D) + power + 40 + math.log2(scale or D ** -0.5) > 129  # of a key of ones
    return c, q


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind,power,scale", FACTORS)
def test_factors_past_32_bits(D, kind, power, scale):
    """Scores of 0, although what they are multiplied with is infinite in 32 bits, beside
    others of -infinity."""
    c, q = past_32_bits(D, [(300, 300), (200, 40)], (0x80, 0x80), kind, power, scale)
    got, status = attend(c, q, softmax_scale=scale)
    assert status == 0
    check(got, *reference(c, q, scale))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("sign", ["any", "negative"])
@pytest.mark.parametrize("kind,size,scale_k", [("f16", 60000.0, -6), ("f16", 60000.0, 0), ("f16", 60000.0, 20), ("f16", 60000.0, 40),
                                               ("bf16", 2.0 ** 40, 0), ("f16", 64.0, 9)])
def test_large_scores(D, sign, kind, size, scale_k):
    """Scores of 2^13 to 2^60, of both signs or all below zero.  A query is one channel of
    the keys, so scores are exact products, equal codes give equal ones, and the largest of a
    row stand apart by a sixteenth of themselves at least."""
    c = Cache([(300, 300), (1100, 50), (17, 1)], 2, D, 32, 16, seed=D + scale_k)
    if sign == "negative":
        for k in (c.codes[0],):
            k.copy_(torch.where(k == 0x7F, k, (k & 0x7F).clamp(0x20, 0x7E) | 0x80))
    c.scales[:, 0] = torch.where(c.scales[:, 0].isnan(), c.scales[:, 0], 2.0 ** scale_k)
    c.scales[:, 1] = torch.where(c.scales[:, 1].isnan(), c.scales[:, 1], 2.0 ** -8)  # (2^z s_V is what is rounded)
    q = torch.zeros(3, 300, 4, D)
    i = torch.arange(300)
    q[:, i, :, i % D] = size
    q[:, ::7] *= 2.0 ** -30 if kind == "bf16" else 2.0 ** -12  # ordinary rows beside them
    q = q.to(KIND[kind][0])
    for b, (_, n) in enumerate(c.lens):
        q[b, n:] = float("nan")
    got, status = attend(c, q)
    assert status == 0
    check(got, *reference(c, q))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("sms", [2, 0])
def test_large_scores_that_come_late(D, sms):
    """Ordinary scores, then some of 2^33, in the rows of one unit: what was summed before
    them is forgotten, in parts of units too."""
    c = Cache([(5000, 200)], 1, D, 64, 64, seed=D)
    c.scales[:, 0] = torch.where(c.scales[:, 0].isnan(), c.scales[:, 0], 2.0 ** -9)
    c.scales[:, 1] = torch.where(c.scales[:, 1].isnan(), c.scales[:, 1], 2.0 ** -8)
    q = torch.zeros(1, 200, 2, D)
    i = torch.arange(200)
    q[:, i, :, i % D] = 8.0
    q[:, 3::5] *= 4096
    for t in (1900, 4400, 4850):
        pg = int(c.table[0, t // 64])
        c.scales[pg, 0] = 2.0 ** 24
    q = q.half()
    got, status = attend(c, q, num_sms=sms)
    assert status == 0
    check(got, *reference(c, q))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind,power,scale", FACTORS)
def test_scores_past_32_bits(D, kind, power, scale):
    """Scores that are +infinity in 32 bits, from a late key on: rows that see it are NaN, the
    others are not concerned."""
    c, q = past_32_bits(D, [(300, 150), (300, 300)], (0, 0x80), kind, power, scale)
    c.codes[0][c.table[0, :6].long()] = 0  # the first such key is 193, the first query that sees it 43
    got, status = attend(c, q, softmax_scale=scale)
    assert status == 0
    ref, tol = reference(c, q, scale)
    assert bool(got[0, 43:150].isnan().all())
    got[0, 43:150] = 0
    ref[0, 43:150] = tol[0, 43:150] = 0
    check(got, ref, tol)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_large_scores_do_not_concern_other_rows(D):
    """Rows of large scores beside ordinary ones in one warp: the others keep their bits."""
    c = Cache([(700, 300)], 1, D, 32, 16, seed=D)
    q = queries(c, 300, 2)
    want, _ = attend(c, q)
    large = torch.rand(300, 2, generator=torch.Generator().manual_seed(D)) < 0.1
    q[0][large] *= 2.0 ** 11
    got, status = attend(c, q)
    assert status == 0
    assert torch.equal(got[0][~large], want[0][~large])
    assert not got.isnan().any() and bool((got[0][large] != want[0][large]).any())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_a_first_key_that_outweighs_all_others(D, kind):
    """The first key has some 2^24 times the weight of any other, and values of zero, so the
    output is the sum of the others, all in one CTA's part of the keys.  The reference of the
    weights goes down to 2^-10 of the first key's after the first step of at most 128 keys
    (there 2^-2): a weight is off by 2^-11 of itself, or by 2^-25 of the reference."""
    L, n = 70000, 40
    c = Cache([(L, n)], 1, D, 64, 64, seed=D)
    g = torch.Generator().manual_seed(D)
    c.codes[0][:] = 0
    pg = c.table[0, :-(-L // 64)].long()
    c.codes[0][pg, :, :, 0] = (torch.randint(0, 0x59, (len(pg), 64, 1), generator=g) + 0x80 *  # up to 16
                               torch.randint(0, 2, (len(pg), 64, 1), generator=g)).to(torch.uint8)
    c.codes[0][pg[0], 0, 0, 0] = 0x7E  # 448
    c.codes[1][pg[0], 0] = 0
    c.codes[1][pg] &= 0x7F  # (sums that do not cancel)
    c.scales = torch.where(c.scales.isnan(), c.scales, torch.ones(()))
    q = torch.zeros(1, n, 2, D)
    q[..., 0] = (0.92 + torch.arange(n) / 250.0)[None, :, None]
    q = q.to(KIND[kind][0])
    scale = 24.5 / 448 / math.log2(math.e)
    ref, _ = reference(c, q, scale)
    got, status = attend(c, q, softmax_scale=scale, num_sms=1)
    assert status == 0
    half = KIND[kind][1]
    (K, _), (V, _) = codes(c, 0, 0), codes(c, 1, 0)
    x = q[0, :, 0, 0].cuda().double()
    z = x[:, None] * K[:, 0, 0] * scale
    z.masked_fill_(torch.arange(L, device="cuda") > (L - n + torch.arange(n, device="cuda"))[:, None], float("-inf"))
    e = torch.exp(z - z.amax(-1, keepdim=True))
    l = e.sum(-1, keepdim=True)
    A = e @ V[:, 0].abs() / l
    small = (2.0 ** -27 * V[:128, 0].abs().sum(0) + 2.0 ** -35 * V[128:, 0].abs().sum(0)) / l  # W = 1: the first key's
    tol = half * ref[0].abs() + (2.0 ** -10 * (A + ref[0, :, 0].abs()) + small)[:, None] + 2.0 ** -25
    assert float(tol.max() / ref[0].max()) < 0.02
    check(got[0], ref[0], tol)


@pytest.mark.parametrize("D,q,G", [(128, 1, 1), (128, 130, 4), (256, 3, 2), (64, 2, 1)])
def test_a_unit_of_seconds(D, q, G):
    """One unit over 2^28 keys on one pair of CTAs takes longer than any wait may.  The first
    4095 entries of its row are one page, whose keys have no weight beside the last one's,
    which are alike: sums of powers of two, of which the output is the value."""
    page, L = 65536, 1 << 28
    k = torch.zeros(2, page, 1, D, dtype=torch.uint8, device="cuda")
    k[0] = 0xFE  # -448
    v = (0x38 + 8 * (torch.arange(D, device="cuda") % 3)).to(torch.uint8).expand(2, page, 1, D).contiguous()  # 1, 2, 4
    bt = torch.zeros(1, L // page, dtype=torch.int32, device="cuda")
    bt[0, -1] = 1
    seq = torch.tensor([[L, q]], dtype=torch.int32, device="cuda")
    x = torch.full((1, q, G, D), 0.25, dtype=torch.float16, device="cuda")
    out = torch.zeros_like(x)
    ws = torch.zeros(vae4.chunk_workspace_bytes(1, G, 1, q, D, L, 2), dtype=torch.uint8, device="cuda")
    vae4.verify_attn_e4m3_chunk(x, k, v, bt, seq, torch.ones(1, 2, device="cuda"), out, ws, num_sms=2)
    torch.cuda.synchronize()
    assert vae4.read_status(ws) == 0
    assert torch.equal(out, v[:1, :1].view(torch.float8_e4m3fn).half().expand_as(out))
