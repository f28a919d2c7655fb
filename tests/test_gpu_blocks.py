"""The block-scaled cache's operators on the GPU against their definitions in
64 bits (torch on the host, sharing no code with the kernels).

Tolerances, derived from the arithmetic:

* append: the codes, scales and bounds are exact (a power-of-two scale makes
  the division exact, so one rounding to 8 bits remains).
* attention: a weight enters the value product rounded to FP16, so off by at
  most 2^-11 of itself (or 2^-25 of the largest, below FP16's normal range);
  the FP32 score of a key is off by far less than 2^-11 in log2 units at these
  sizes, which the factor 2 in 2^-10 covers together with the FP32 sums; the
  output is rounded once to FP16.  With A = sum p |V| and n keys:
      |got - out| <= 2^-11 |out| + 2^-10 (A + |out|) + n 2^-25 max|V| + 2^-24
* scores: FP32 sums of 2D exact products: 2D * 2^-24 of the sum of magnitudes.
* choices of blocks: exact.
"""
import math

import pytest
import torch

import fp8_paged_attention_e4m3_gb300 as vae4

pytestmark = pytest.mark.gpu

FMT = {"e4m3": (torch.float8_e4m3fn, 448.0, 0), "e5m2": (torch.float8_e5m2, 57344.0, vae4.FLAG_KV_E5M2)}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    vae4.load()


def dev(*ts):
    return [t.cuda() if t is not None else None for t in ts]


class Cache:
    """A paged block-scaled cache of random values on the host: K and V as
    [n_pages][page][Hkv][D] bytes, scales, block table and lengths.  Every
    slot that no sequence's token occupies holds a NaN code, and every scale
    of a block without tokens is NaN."""

    def __init__(self, lens, Hkv, D, page, blk, fmt="e4m3", seed=0, spread=1.0, extra=3):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.Hkv, self.D, self.page, self.blk, self.fmt = lens, Hkv, D, page, blk, fmt
        kind, top, _ = FMT[fmt]
        nb = page // blk
        per = [-(-L // page) for L, _ in lens]
        self.n_pages = sum(per) + extra
        order = torch.randperm(self.n_pages, generator=g).int()
        self.table = torch.full((len(lens), max(max(per), 1) + 1), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(per):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.codes, self.scales = [], torch.full((self.n_pages, 2, Hkv, nb), float("nan"))
        for w in (0, 1):
            x = torch.randn(self.n_pages, nb, blk, Hkv, D, generator=g)
            x *= torch.exp2(spread * torch.randn(self.n_pages, nb, 1, Hkv, 1, generator=g))
            sc = x.abs().amax((2, 4)) / top
            self.scales[:, w] = sc.transpose(1, 2)
            y = (x / sc[:, :, None, :, None]).clamp(-top, top).to(kind).view(torch.uint8)
            self.codes.append(y.reshape(self.n_pages, page, Hkv, D))
        live = torch.zeros(self.n_pages, page, dtype=torch.bool)
        for b, (L, _) in enumerate(lens):
            for j in range(per[b]):
                live[self.table[b, j], :max(0, min(page, L - j * page))] = True
        for c in self.codes:
            c[~live] = 0x7F
        dead = ~live.view(self.n_pages, nb, blk).any(-1)  # [n_pages][nb]
        self.scales[dead[:, None, None].expand_as(self.scales)] = float("nan")
        self.seq = torch.tensor(lens, dtype=torch.int32)

    def values(self, w, b):
        """The L values [L][Hkv][D] of K (0) or V (1) of sequence b in 64 bits."""
        L = self.lens[b][0]
        pg = self.table[b, :-(-L // self.page)].long()
        x = self.codes[w][pg].view(FMT[self.fmt][0]).double()
        s = self.scales[pg, w].double().repeat_interleave(self.blk, 2).transpose(1, 2)
        return (x * s[..., None]).flatten(0, 1)[:L]

    def device(self, layout="tokens"):
        """(K, V) on the device: token-major, the pool's views, or token-major
        with a token stride of 8 (not 16) bytes' granularity."""
        n, page, H, D = self.codes[0].shape
        if layout == "pool":
            kv = torch.stack([c.transpose(1, 2) for c in self.codes], 1).contiguous().cuda()
            return vae4.cache_views(kv)
        if layout == "padded":
            out = []
            for c in self.codes:
                buf = torch.full((n, page, H * D + 8), 0x7F, dtype=torch.uint8, device="cuda")
                view = buf[:, :, :H * D].unflatten(2, (H, D))
                view.copy_(c)
                out.append(view)
            return tuple(out)
        return tuple(dev(*self.codes))


def reference(c, q, scale=0.0, allowed=None):
    """(out, bound) in 64 bits; allowed(b, i, h, pos): the keys the query may see."""
    B, Q, Hq, D = q.shape
    G = Hq // c.Hkv
    sm = scale or 1 / math.sqrt(D)
    out = torch.zeros(B, Q, Hq, D, dtype=torch.float64)
    tol = torch.zeros_like(out)
    for b, (L, n) in enumerate(c.lens):
        if L == 0:
            continue
        K, V = c.values(0, b), c.values(1, b)
        for i in range(n):
            seen = torch.arange(L - n + i + 1)
            for h in range(c.Hkv):
                keep = seen if allowed is None else allowed(b, i, h, L - n + i)
                if keep.numel() == 0:
                    continue
                z = q[b, i, h * G:(h + 1) * G].double() @ K[keep, h].T * sm
                p = torch.softmax(z, -1)
                o = p @ V[keep, h]
                a = p @ V[keep, h].abs()
                out[b, i, h * G:(h + 1) * G] = o
                tol[b, i, h * G:(h + 1) * G] = (2.0 ** -11 * o.abs() + 2.0 ** -10 * (a + o.abs()) +
                                                keep.numel() * 2.0 ** -25 * V[keep, h].abs().max() +
                                                2.0 ** -24)
    return out, tol


def queries(c, Q, G, seed=1):
    """FP16 queries; the padding slots hold NaN."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(len(c.lens), Q, G * c.Hkv, c.D, generator=g).half()
    for b, (_, n) in enumerate(c.lens):
        q[b, n:] = float("nan")
    return q


def attend(c, q, layout="tokens", **kw):
    B, Q, Hq, D = q.shape
    cap = kw.pop("max_seq_len", 0)
    k, v = c.device(layout)
    qd, bt, seq, sc = dev(q, c.table, c.seq, c.scales)
    out = torch.full_like(qd, float("nan"))
    top = cap or c.table.shape[1] * c.page
    n = vae4.block_scaled_workspace_bytes(B, Hq, c.Hkv, Q, D, top, kw.get("num_sms", 0))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    vae4.verify_attn_e4m3_block_scaled(qd, k, v, bt, seq, sc, out, ws, max_seq_len=cap,
                                       flags=FMT[c.fmt][2], **kw)
    torch.cuda.synchronize()
    return out.cpu(), vae4.read_status(ws)


def check(got, ref, tol):
    got = got.double()
    assert torch.isfinite(got).all()
    far = ((got - ref).abs() - tol).max().item()
    assert far <= 0, f"{far} past the bound; largest difference {(got - ref).abs().max().item()}"


ATTEND = [
    # lens, Q, G, Hkv, D, page, block, format, layout
    ([(1, 1)], 1, 1, 1, 64, 16, 16, "e4m3", "tokens"),
    ([(17, 8)], 8, 2, 1, 64, 16, 16, "e4m3", "pool"),
    ([(1024, 8)], 8, 2, 1, 64, 16, 16, "e4m3", "tokens"),
    ([(3297, 8), (1025, 5), (0, 0), (16, 16), (15, 1)], 16, 6, 1, 256, 16, 16, "e4m3", "tokens"),
    ([(700, 16), (3000, 16)], 16, 6, 1, 256, 48, 48, "e4m3", "pool"),
    ([(2500, 1), (95, 1), (96, 1), (97, 1)], 1, 8, 4, 128, 96, 32, "e4m3", "tokens"),
    ([(2500, 3), (777, 2)], 5, 4, 3, 128, 64, 64, "e5m2", "pool"),
    ([(5000, 8)], 8, 6, 1, 256, 848, 848, "e4m3", "padded"),
    ([(1500, 8), (300, 8)], 8, 4, 2, 128, 32, 16, "e4m3", "padded"),
    ([(4000, 4)], 4, 12, 2, 64, 128, 16, "e5m2", "padded"),
    ([(300, 2)] * 40, 2, 3, 2, 64, 32, 32, "e4m3", "tokens"),
    # several units per SM, in one and in several batches of segments
    ([(200 + 37 * b, 1) for b in range(30)], 1, 16, 8, 128, 64, 32, "e4m3", "tokens"),
    ([(70, 4)] * 33, 4, 12, 2, 256, 64, 64, "e4m3", "pool"),
    ([(9000, 1)] + [(5, 1)] * 900, 1, 2, 2, 64, 16, 16, "e4m3", "tokens"),
    ([(20, 1)] * 1500, 1, 1, 8, 64, 32, 32, "e4m3", "tokens"),
    # more sequences than the plan stages
    ([(1 + b % 40, 1) for b in range(4500)], 1, 2, 1, 64, 16, 16, "e4m3", "tokens"),
]


@pytest.mark.parametrize("lens,Q,G,Hkv,D,page,blk,fmt,layout", ATTEND,
                         ids=[f"{len(c[0])}x{c[3]}-q{c[1]}x{c[2]}-{c[4]}-{c[5]}/{c[6]}-{c[7]}-{c[8]}"
                              for c in ATTEND])
def test_attention_matches_the_definition(lens, Q, G, Hkv, D, page, blk, fmt, layout):
    c = Cache(lens, Hkv, D, page, blk, fmt, seed=len(lens) + D)
    q = queries(c, Q, G)
    got, status = attend(c, q, layout)
    assert status == 0
    check(got, *reference(c, q))
    for b, (L, n) in enumerate(lens):  # padding slots and dead sequences
        assert not got[b, n if L else 0:].any()


@pytest.mark.parametrize("sms", [1, 3, 152, 400])
def test_attention_divided_among_other_numbers_of_sms(sms):
    """Fewer CTAs than units (one CTA walks them all) and more than the GPU's
    SMs; the same call twice gives the same bits."""
    c = Cache([(1000, 3), (130, 1), (64, 2), (2000, 3), (0, 0), (700, 2)], 2, 128, 32, 16, seed=12)
    q = queries(c, 3, 4)
    got, status = attend(c, q, num_sms=sms)
    assert status == 0
    check(got, *reference(c, q))
    again, _ = attend(c, q, num_sms=sms)
    assert torch.equal(got, again)


def test_attention_over_more_parts_than_the_combine_holds():
    """num_sms beyond 4096 counts as 4096."""
    c = Cache([(420000, 1)], 1, 64, 64, 64, seed=14)
    q = queries(c, 1, 2)
    got, status = attend(c, q, num_sms=10000)
    assert status == 0
    check(got, *reference(c, q))
    again, _ = attend(c, q, num_sms=4096)
    assert torch.equal(got, again)


def test_calls_at_once_on_two_streams():
    """Calls on two streams, each with its own workspace and outputs, give what
    they give alone."""
    c = Cache([(6000, 2), (900, 3), (3100, 1)], 2, 128, 32, 16, seed=15)
    q = queries(c, 3, 4)
    k, v = c.device()
    qd, bt, seq, sc = dev(q, c.table, c.seq, c.scales)
    ids = random_ids(c, 3, 40).cuda()
    cap = c.table.shape[1] * c.page
    outs = [torch.empty(12, *qd.shape, dtype=torch.float16, device="cuda") for _ in range(4)]
    ws = [vae4.alloc_workspace(3, 8, 2, 3, 128, cap), vae4.alloc_sparse_workspace(3, 8, 2, 3, 128, cap, 16, 40)]
    ws += [w.clone() for w in ws]

    def both(o, w, n, stream):
        for x in range(n):
            vae4.verify_attn_e4m3_block_scaled(qd, k, v, bt, seq, sc, o[0][x], w[0], stream=stream)
            vae4.verify_attn_e4m3_sparse(qd, k, v, bt, seq, sc, ids, o[1][x], w[1], stream=stream)

    both(outs[:2], ws[:2], 1, None)
    torch.cuda.synchronize()
    want = [outs[0][0].clone(), outs[1][0].clone()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for o in outs:
        o.fill_(float("nan"))
    torch.cuda.synchronize()
    both(outs[:2], ws[:2], 12, streams[0])
    both(outs[2:], ws[2:], 12, streams[1])
    torch.cuda.synchronize()
    for e, o in enumerate(outs):
        assert (o == want[e % 2]).all()
    assert all(vae4.read_status(w) == 0 for w in ws)


def test_waits_that_run_out_mark_the_rows():
    """The failure path: every pipeline wait gives up at once, the call reports
    the timeout and writes zero rows, and the workspace serves the next call."""
    c = Cache([(3000, 4), (100, 4), (50, 2)], 2, 128, 32, 16, seed=13)
    q = queries(c, 4, 3)
    k, v = c.device()
    qd, bt, seq, sc = dev(q, c.table, c.seq, c.scales)
    ids = torch.arange(6, dtype=torch.int32).expand(3, 4, 2, 6).contiguous().cuda()
    cap = c.table.shape[1] * c.page
    for sp in (False, True):
        ws = (vae4.alloc_sparse_workspace(3, 6, 2, 4, 128, cap, 16, 6) if sp else
              vae4.alloc_workspace(3, 6, 2, 4, 128, cap))
        out = torch.full_like(qd, float("nan"))
        for flags in (vae4.FLAG_TEST_SHORT_WAITS, 0):
            if sp:
                vae4.verify_attn_e4m3_sparse(qd, k, v, bt, seq, sc, ids, out, ws, flags=flags)
            else:
                vae4.verify_attn_e4m3_block_scaled(qd, k, v, bt, seq, sc, out, ws, flags=flags)
            torch.cuda.synchronize()
            assert vae4.read_status(ws) == (vae4.STATUS_TIMEOUT if flags else 0)
            if flags:
                assert not out.any()
                vae4.clear_status(ws)
        allowed = listed(c, ids.cpu()) if sp else None
        check(out.cpu(), *reference(c, q, allowed=allowed))


def test_attention_with_scales_far_apart():
    """Blocks whose V scales differ by up to 2^40: the weights carry s_V, the
    running sum does not, and neither overflows nor loses the small blocks'
    share."""
    c = Cache([(640, 4)], 2, 128, 64, 16, seed=5)
    g = torch.Generator().manual_seed(9)
    e = torch.randint(-20, 21, c.scales[:, 1].shape, generator=g)
    e[int(c.table[0, 0])], e[int(c.table[0, 1])] = -20, 20
    c.scales[:, 1] = torch.where(c.scales[:, 1].isnan(), c.scales[:, 1], torch.exp2(e.float() - 18))
    q = queries(c, 4, 3)
    ref, tol = reference(c, q)
    assert ref.abs().max() < 6e4
    got, status = attend(c, q)
    assert status == 0
    check(got, ref, tol)


def test_attention_lengths_without_q_and_softmax_scale():
    c = Cache([(100, 3), (40, 3)], 1, 64, 32, 16, seed=3)
    q = queries(c, 3, 5)
    c.seq = torch.tensor([100, 40], dtype=torch.int32)  # q = Qmax for all
    got, status = attend(c, q, softmax_scale=0.31)
    assert status == 0
    check(got, *reference(c, q, 0.31))


def test_invalid_pages_scales_and_lengths():
    lens = [(200, 2), (300, 2), (250, 2), (90, 2)]
    c = Cache(lens, 2, 64, 32, 16, seed=4)
    q = queries(c, 2, 2)
    ref, tol = reference(c, q)
    c.table[0, 2] = c.n_pages            # sequence 0: a page past the pool
    pg = int(c.table[1, 3])
    c.scales[pg, 1, 1, 0] = float("inf")  # sequence 1, KV head 1: an invalid V scale
    c.seq[2, 0] = 100000                 # sequence 2: longer than the table
    got, status = attend(c, q)
    assert status == vae4.STATUS_BAD_BLOCK | vae4.STATUS_BAD_SCALE | vae4.STATUS_BAD_LENGTH
    ref[0] = tol[0] = 0
    ref[1, :, 2:] = tol[1, :, 2:] = 0
    ref[2] = tol[2] = 0
    check(got, ref, tol)
    for bad in (0.0, -1.0, float("nan"), 2.0 ** 41, 2.0 ** -41):
        c2 = Cache(lens[:1], 1, 64, 32, 16, seed=4)
        c2.scales[int(c2.table[0, 1]), 0, 0, 1] = bad
        got, status = attend(c2, queries(c2, 2, 2))
        assert status == vae4.STATUS_BAD_SCALE and not got.any()


# ------------------------------------------------------------------ sparse
def sparse(c, q, ids, layout="tokens", **kw):
    B, Q, Hq, D = q.shape
    k, v = c.device(layout)
    qd, bt, seq, sc, idd = dev(q, c.table, c.seq, c.scales, ids)
    out = torch.full_like(qd, float("nan"))
    ws = vae4.alloc_sparse_workspace(B, Hq, c.Hkv, Q, D, c.table.shape[1] * c.page, c.blk, ids.shape[3])
    vae4.verify_attn_e4m3_sparse(qd, k, v, bt, seq, sc, idd, out, ws, flags=FMT[c.fmt][2], **kw)
    torch.cuda.synchronize()
    return out.cpu(), vae4.read_status(ws)


def listed(c, ids):
    def allowed(b, i, h, pos):
        keys = [t for j in sorted(set(ids[b, i, h].tolist())) if j >= 0
                for t in range(j * c.blk, min((j + 1) * c.blk, pos + 1))]
        return torch.tensor(keys, dtype=torch.long)
    return allowed


def random_ids(c, Q, k, seed=2):
    """Lists with repetitions, in no order, some entries out of range and some
    lists empty."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.full((len(c.lens), Q, c.Hkv, k), -1, dtype=torch.int32)
    for b, (L, n) in enumerate(c.lens):
        nblk = -(-L // c.blk)
        if nblk == 0:
            continue
        shared = torch.randint(0, nblk, (c.Hkv, k), generator=g)
        for i in range(n):
            mine = torch.randint(-2, nblk + 2, (c.Hkv, k), generator=g)
            pick = torch.rand(c.Hkv, k, generator=g) < 0.6
            ids[b, i] = torch.where(pick, shared, mine).int()
    ids[0, 0, 0] = -1  # an empty set
    ids[-1, -1, -1] = 1 << 30
    return ids


SPARSE = [
    ([(1, 1)], 1, 1, 1, 64, 16, 16, 1, "e4m3", "tokens"),
    ([(1000, 1)], 1, 6, 2, 256, 16, 16, 9, "e4m3", "tokens"),
    ([(2000, 8), (999, 5), (0, 0), (17, 8)], 8, 6, 1, 256, 16, 16, 12, "e4m3", "pool"),
    ([(3000, 16), (500, 3)], 16, 6, 2, 128, 96, 48, 7, "e4m3", "tokens"),
    ([(2049, 1), (64, 1), (63, 1), (700, 1)], 1, 8, 4, 128, 64, 64, 6, "e5m2", "pool"),
    ([(1200, 4), (800, 4)], 4, 3, 2, 64, 48, 16, 10, "e4m3", "padded"),
    ([(600, 2)] * 50, 2, 2, 3, 64, 32, 32, 4, "e4m3", "tokens"),
    ([(40, 1)] * 520, 1, 1, 2, 64, 16, 16, 2, "e4m3", "tokens"),   # more than 1024 streams
    ([(1 + b % 70, 1) for b in range(2100)], 1, 1, 2, 64, 16, 16, 2, "e4m3", "tokens"),  # 4200
    ([(5000, 2)], 2, 4, 1, 128, 848, 848, 3, "e4m3", "tokens"),
    ([(5000, 2)], 2, 4, 1, 128, 848, 848, 3, "e4m3", "padded"),
    ([(4000, 3)], 3, 4, 1, 256, 32, 16, 200, "e4m3", "pool"),      # one stream over many SMs
]


@pytest.mark.parametrize("lens,Q,G,Hkv,D,page,blk,k,fmt,layout", SPARSE)
def test_sparse_matches_the_definition(lens, Q, G, Hkv, D, page, blk, k, fmt, layout):
    c = Cache(lens, Hkv, D, page, blk, fmt, seed=len(lens) + D)
    q = queries(c, Q, G)
    ids = random_ids(c, Q, k)
    got, status = sparse(c, q, ids, layout)
    assert status == 0
    check(got, *reference(c, q, allowed=listed(c, ids)))


def test_sparse_with_every_block_is_the_whole_attention():
    c = Cache([(777, 8), (320, 8)], 2, 128, 32, 16, seed=6)
    q = queries(c, 8, 3)
    ids = torch.arange(49, dtype=torch.int32).expand(2, 8, 2, 49).contiguous()
    got, status = sparse(c, q, ids)
    assert status == 0
    check(got, *reference(c, q))


def test_sparse_reads_the_listed_blocks_alone():
    """Blocks in no list: NaN codes, invalid scales and pages do no harm.  An
    invalid page or scale of a listed block zeroes its sequence and head."""
    lens = [(512, 2), (512, 2)]
    c = Cache(lens, 2, 64, 16, 16, seed=7)
    q = queries(c, 2, 2)
    ids = torch.tensor([1, 5, 31, -1], dtype=torch.int32).expand(2, 2, 2, 4).contiguous()
    ids[:, 1, :, 3] = 8
    ref, tol = reference(c, q, allowed=listed(c, ids))
    used = {1, 5, 8, 31}
    for b in range(2):
        for j in range(32):
            if j not in used:
                pg = int(c.table[b, j])
                for code in c.codes:
                    code[pg] = 0x7F
                c.scales[pg] = float("nan")
                if j % 2:
                    c.table[b, j] = -5
    got, status = sparse(c, q, ids)
    assert status == 0
    check(got, ref, tol)
    c.table[0, 5] = c.n_pages
    c.scales[int(c.table[1, 8]), 0, 0] = -1
    got, status = sparse(c, q, ids)
    assert status == vae4.STATUS_BAD_BLOCK | vae4.STATUS_BAD_SCALE
    ref[0] = tol[0] = 0
    ref[1, :, :2] = tol[1, :, :2] = 0
    check(got, ref, tol)


# ------------------------------------------------------------------ scores
def bounds_of(c):
    """Bounds of K of every block that holds tokens, as codes."""
    nb = c.page // c.blk
    kind = FMT[c.fmt][0]
    bd = torch.full((c.n_pages, c.Hkv, nb, 2, c.D), 0x7F, dtype=torch.uint8)
    for b, (L, _) in enumerate(c.lens):
        for j in range(-(-L // c.blk)):
            pg, slot = int(c.table[b, j * c.blk // c.page]), j * c.blk % c.page
            x = c.codes[0][pg, slot:slot + min(c.blk, L - j * c.blk)].view(kind).float()
            bd[pg, :, slot // c.blk] = torch.stack([x.amin(0), x.amax(0)], 1).to(kind).view(torch.uint8)
    return bd


SCORES = [
    ([(1, 1)], 1, 1, 1, 64, 16, 16, "e4m3"),
    ([(1000, 8), (333, 3), (0, 0)], 8, 6, 2, 256, 64, 16, "e4m3"),
    ([(2000, 16)], 16, 6, 1, 128, 32, 32, "e4m3"),
    ([(3000, 1), (65, 1)], 1, 16, 2, 128, 96, 48, "e5m2"),
    ([(4100, 5), (4095, 2)], 5, 5, 3, 64, 16, 16, "e4m3"),
    ([(700, 2)] * 9, 3, 7, 1, 256, 128, 64, "e4m3"),
]


@pytest.mark.parametrize("lens,Q,G,Hkv,D,page,blk,fmt", SCORES)
def test_scores_match_the_definition(lens, Q, G, Hkv, D, page, blk, fmt):
    c = Cache(lens, Hkv, D, page, blk, fmt, seed=len(lens) + D)
    q, bd = queries(c, Q, G), bounds_of(c)
    cols = max(-(-L // blk) for L, _ in lens) + 2
    qd, bdd, bt, seq, sc = dev(q, bd, c.table, c.seq, c.scales)
    got = torch.full((len(lens), Q, Hkv, cols), 123.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    vae4.verify_attn_e4m3_block_scores(qd, bdd, bt, seq, sc, got, block_tokens=blk, status=status,
                                       flags=FMT[fmt][2])
    got = got.cpu().double()
    assert int(status) == 0
    for b, (L, n) in enumerate(lens):
        nblk = -(-L // blk)
        assert (got[b, n:] == 123).all() and (got[b, :, :, nblk:] == 123).all()  # left as they were
        if nblk == 0:
            continue
        j = torch.arange(nblk)
        pg, sub = c.table[b, j * blk // page].long(), j * blk % page // blk
        lohi = bd[pg, :, sub].view(FMT[fmt][0]).double()  # [nblk][H][2][D]
        s = c.scales[pg, 0, :, sub].double() / math.sqrt(D)  # [nblk][H]
        K = c.values(0, b)
        for i in range(n):
            qq = q[b, i].double().view(Hkv, G, D)
            terms = torch.maximum(qq * lohi[:, :, None, 0], qq * lohi[:, :, None, 1])
            want = terms.sum(-1).amax(-1) * s  # [nblk][H]
            mags = torch.maximum((qq * lohi[:, :, None, 0]).abs(), (qq * lohi[:, :, None, 1]).abs())
            tol = (2 * D + 4) * 2.0 ** -24 * mags.sum(-1).amax(-1) * s
            hidden = j * blk > L - n + i
            g = got[b, i, :, :nblk].T
            assert (g[hidden] == -math.inf).all()
            assert ((g - want).abs() <= tol)[~hidden].all()
            for jj in range(min(3, nblk)):  # it bounds the block's logits
                z = torch.einsum("hgd,thd->hgt", qq, K[jj * blk:(jj + 1) * blk]) / math.sqrt(D)
                assert (z.amax((1, 2)) <= want[jj] + tol[jj]).all()


def test_scores_report_pages_and_columns():
    c = Cache([(160, 1), (300, 1)], 1, 64, 16, 16, seed=3)
    q, bd = queries(c, 1, 2), bounds_of(c)
    c.table[0, 4] = -1
    qd, bdd, bt, seq, sc = dev(q, bd, c.table, c.seq, c.scales)
    got = torch.full((2, 1, 1, 10), 7.0, device="cuda")  # 19 blocks of sequence 1 do not fit
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    vae4.verify_attn_e4m3_block_scores(qd, bdd, bt, seq, sc, got, block_tokens=16, status=status)
    assert int(status) == vae4.STATUS_BAD_BLOCK | vae4.STATUS_BAD_LENGTH
    assert (got[1] == 7).all() and got[0, 0, 0, 4] == -math.inf
    assert torch.isfinite(got[0, 0, 0, [0, 1, 2, 3, 5, 6, 7, 8, 9]]).all()


@pytest.mark.parametrize("B,Q,G,Hkv,D,nblk", [
    (2, 3, 2, 8, 64, 1400), (1, 16, 6, 2, 128, 6000), (40, 1, 8, 8, 128, 520), (1, 7, 12, 1, 256, 700),
    (1, 5, 3, 4, 64, 2600),
])
def test_scores_of_many_blocks(B, Q, G, Hkv, D, nblk):
    """Grids in which queries share CTAs or not, and warps take several steps."""
    g = torch.Generator(device="cuda").manual_seed(nblk)
    blk = 16
    lens = [(max(1, nblk * blk - 1 - 977 * b % (nblk * blk)), 1 + (Q - 1) * (b + 1) // B) for b in range(B)]
    lens = [(L, min(n, L)) for L, n in lens]
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    table = torch.randperm(B * nblk, generator=g, device="cuda").int().view(B, nblk)
    x = torch.randn(B * nblk, Hkv, 1, 2, D, generator=g, device="cuda").sort(3).values
    bd = x.to(torch.float8_e4m3fn).view(torch.uint8)
    sc = torch.exp2(torch.randint(-3, 4, (B * nblk, 2, Hkv, 1), generator=g, device="cuda").float())
    q = torch.randn(B, Q, G * Hkv, D, generator=g, device="cuda").half()
    got = torch.full((B, Q, Hkv, nblk), 7.0, device="cuda")
    vae4.verify_attn_e4m3_block_scores(q, bd, table, seq, sc, got, block_tokens=blk)
    for b, (L, n) in enumerate(lens):
        v = (L - 1) // blk + 1
        pg = table[b, :v].long()
        lohi = bd[pg, :, 0].view(torch.float8_e4m3fn).double()  # [v][H][2][D]
        s = sc[pg, 0, :, 0].double() / math.sqrt(D)
        assert (got[b, n:] == 7).all() and (got[b, :, :, v:] == 7).all()  # left as they were
        for i in range(n):
            qq = q[b, i].double().view(Hkv, G, D)
            want = (torch.einsum("hgd,vhd->vhg", qq.clamp(min=0), lohi[:, :, 1]) +
                    torch.einsum("hgd,vhd->vhg", qq.clamp(max=0), lohi[:, :, 0])).amax(-1) * s
            mags = torch.einsum("hgd,vhd->vhg", qq.abs(), lohi.abs().amax(2)).amax(-1) * s
            hidden = torch.arange(v, device="cuda") * blk > L - n + i
            r = got[b, i, :, :v].T.double()
            assert (r[hidden] == -math.inf).all()
            assert ((r - want).abs() <= (2 * D + 4) * 2.0 ** -24 * mags)[~hidden].all()


# ------------------------------------------------------------------ choice of blocks
def choose(row, v, k, sink, local):
    if v <= k:
        ids = list(range(v))
    else:
        key = [(-math.inf if math.isnan(x) else x + 0.0) for x in row[:v]]
        cand = sorted(range(sink, v - local), key=lambda j: (-key[j], j))
        ids = sorted(list(range(sink)) + list(range(v - local, v)) + cand[:k - sink - local])
    return ids + [-1] * (k - len(ids))


@pytest.mark.parametrize("L,q,blk,k,sink,local,kind", [
    (1, 1, 16, 1, 0, 1, "plain"), (100, 4, 16, 7, 0, 0, "plain"), (100, 4, 16, 8, 1, 1, "plain"),
    (5000, 8, 16, 17, 2, 3, "plain"), (5000, 8, 16, 40, 0, 0, "ties"), (5000, 2, 16, 5, 3, 2, "ties"),
    (9000, 3, 16, 64, 1, 1, "odd"), (20000, 2, 16, 300, 4, 4, "odd"), (9000, 2, 16, 33, 0, 0, "equal"),
    (1600000, 1, 16, 100, 1, 2, "plain"), (1000000, 1, 16, 2000, 0, 1, "ties"),
    (70000, 1, 64, 1093, 0, 1, "plain"), (33333, 16, 48, 25, 1, 1, "close"),
])
def test_choice_of_blocks(L, q, blk, k, sink, local, kind):
    g = torch.Generator().manual_seed(L + k)
    lens = [(L, q), (max(q, L // 3), max(1, q - 1)), (0, 0)]
    n = -(-L // blk) + 3
    x = torch.randn(3, q, 2, n, generator=g)
    if kind == "ties":
        x = x.round()
        x[torch.rand(x.shape, generator=g) < 0.3] = -0.0
    elif kind == "odd":
        r = torch.rand(x.shape, generator=g)
        x[r < 0.02] = float("nan")
        x[(r >= 0.02) & (r < 0.04)] = float("inf")
        x[(r >= 0.04) & (r < 0.5)] = -float("inf")
        x[(r >= 0.5) & (r < 0.55)] = 1e-42
    elif kind == "equal":
        x[:] = -2.5
    elif kind == "close":
        x = 1 + x * 1e-6
    wide = torch.zeros(3, q, 2, n + 5, device="cuda")  # rows that are not contiguous
    wide[..., :n] = x
    ids = torch.full((3, q, 2, k), -9, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    vae4.verify_attn_e4m3_select_blocks(wide[..., :n], seq, ids, block_tokens=blk, sink_blocks=sink,
                                        local_blocks=local, status=status)
    ids = ids.cpu()
    assert int(status) == 0
    for b, (Lb, nb) in enumerate(lens):
        for i in range(q):
            for h in range(2):
                v = (Lb - nb + i) // blk + 1 if Lb and i < nb else 0
                assert ids[b, i, h].tolist() == choose(x[b, i, h].tolist(), v, k, sink, local), (b, i, h)


def test_choice_reports_lengths():
    x = torch.zeros(3, 1, 1, 4, device="cuda")
    ids = torch.zeros(3, 1, 1, 3, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    seq = torch.tensor([[65, 1], [64, 1], [5, 6]], dtype=torch.int32, device="cuda")
    vae4.verify_attn_e4m3_select_blocks(x, seq, ids, block_tokens=16, status=status)
    assert int(status) == vae4.STATUS_BAD_LENGTH | vae4.STATUS_BAD_QLEN
    assert ids[:, 0, 0].tolist() == [[-1, -1, -1], [0, 1, 3], [-1, -1, -1]]


# ------------------------------------------------------------------ append
def pow2_for(a, top):
    if a == 0:
        return 2.0 ** -30
    e = math.frexp(a / top)[1] - 1
    while top * 2.0 ** e < a:
        e += 1
    while top * 2.0 ** (e - 1) >= a:
        e -= 1
    return 2.0 ** min(max(e, -30), 30)


def append_reference(c, k_new, v_new, codes, scales, bounds):
    """The definition, block by block; returns the status bits."""
    kind, top, _ = FMT[c.fmt]
    status = 0
    for b, (L, n) in enumerate(c.lens):
        if n == 0:
            continue
        for j in range((L - n) // c.blk, -(-L // c.blk)):
            t0 = j * c.blk
            pg, slot, sub = int(c.table[b, t0 // c.page]), t0 % c.page, t0 % c.page // c.blk
            a, z = max(0, L - n - t0), min(c.blk, L - t0)
            for w, new in ((0, k_new), (1, v_new)):
                x = new[b, t0 + a - (L - n):t0 + z - (L - n)].double()  # [t][H][D]
                for h in range(c.Hkv):
                    xh = x[:, h]
                    fin = xh[torch.isfinite(xh)].abs()
                    need = pow2_for(float(fin.max()) if fin.numel() else 0.0, top)
                    if not torch.isfinite(xh).all() or (fin.numel() and fin.max() > top * 2.0 ** 30):
                        status |= vae4.STATUS_BAD_VALUE
                    old = float(scales[pg, w, h, sub])
                    s = max(old, need) if a else need
                    y = codes[w][pg, slot:slot + a, h].view(kind).double()
                    y = torch.cat([y * (old / s) if a else y,
                                   (torch.nan_to_num(xh, nan=0.0, posinf=1e300, neginf=-1e300) / s)])
                    y = y.clamp(-top, top).float().to(kind)
                    codes[w][pg, slot:slot + z, h] = y.view(torch.uint8)
                    scales[pg, w, h, sub] = s
                    if w == 0 and bounds is not None:
                        f = y.float()
                        bounds[pg, h, sub] = torch.stack([f.amin(0), f.amax(0)]).to(kind).view(torch.uint8)
    return status


def same_values(a, b, kind):
    return torch.equal(a.contiguous().view(kind).float().nan_to_num(1e9),
                       b.contiguous().view(kind).float().nan_to_num(1e9))


APPEND = [
    # lens, Qmax, Hkv, D, page, block, format, layout, type, bounds
    ([(1, 1)], 1, 1, 64, 16, 16, "e4m3", "tokens", torch.float16, True),
    ([(101, 1), (16, 1), (17, 1), (32, 1)], 1, 2, 64, 16, 16, "e4m3", "pool", torch.float16, True),
    ([(101, 8), (300, 5), (0, 0), (8, 8), (48, 0)], 8, 2, 256, 16, 16, "e4m3", "tokens", torch.float16, True),
    ([(700, 333), (64, 64), (65, 65), (321, 1)], 333, 3, 128, 64, 64, "e4m3", "pool", torch.bfloat16, True),
    ([(1000, 900)], 900, 1, 64, 848, 848, "e4m3", "tokens", torch.float16, True),
    ([(97, 40), (49, 2)], 40, 2, 128, 96, 48, "e5m2", "tokens", torch.bfloat16, True),
    ([(97, 40), (49, 2)], 41, 2, 256, 48, 16, "e4m3", "padded", torch.bfloat16, False),
    ([(2500, 2500)], 2500, 2, 256, 128, 128, "e5m2", "pool", torch.float16, False),
]


def run_append(c, k_new, v_new, layout, bounds, status, kv=None, sc=None, bd=None):
    k, v = kv if kv else c.device(layout)
    sc = c.scales.cuda() if sc is None else sc
    kd, vd, bt, seq = dev(k_new, v_new, c.table, c.seq)
    if bounds and bd is None:
        bd = torch.full((c.n_pages, c.Hkv, c.page // c.blk, 2, c.D), 0x3C, dtype=torch.uint8, device="cuda")
    vae4.verify_attn_e4m3_append(kd, vd, k, v, bt, seq, sc, k_bounds=bd, status=status,
                                 flags=FMT[c.fmt][2])
    torch.cuda.synchronize()
    return (k, v), sc, bd


@pytest.mark.parametrize("lens,Q,Hkv,D,page,blk,fmt,layout,dtype,bounds", APPEND)
def test_append_matches_the_definition(lens, Q, Hkv, D, page, blk, fmt, layout, dtype, bounds):
    c = Cache(lens, Hkv, D, page, blk, fmt, seed=D + Q)
    c.scales = torch.exp2(c.scales.log2().round())  # as earlier calls left them
    g = torch.Generator().manual_seed(Q)
    shape = (len(lens), Q, Hkv, D)
    k_new, v_new = [(torch.randn(shape, generator=g) *
                     torch.exp2(3 * torch.randn(len(lens), Q, Hkv, 1, generator=g))).to(dtype)
                    for _ in range(2)]
    for b, (_, n) in enumerate(lens):
        k_new[b, n:] = float("nan")  # padding is not read
    codes, scales = [x.clone() for x in c.codes], c.scales.clone()
    kind = FMT[fmt][0]
    bd = torch.full((c.n_pages, Hkv, page // blk, 2, D), 0x3C, dtype=torch.uint8) if bounds else None
    assert append_reference(c, k_new, v_new, codes, scales, bd) == 0
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv, sc, bdd = run_append(c, k_new, v_new, layout, bounds, status)
    for again in range(2):  # and once more: nothing changes
        assert int(status) == 0
        assert torch.equal(sc.cpu().nan_to_num(-1), scales.nan_to_num(-1))
        for got, want in zip(kv, codes):
            assert same_values(got.cpu(), want, kind)
        if bounds:
            assert same_values(bdd.cpu(), bd, kind)
        run_append(c, k_new, v_new, layout, bounds, status, kv, sc, bdd)


def test_append_values_at_the_edges():
    """Zeros, the largest value of a scale and the next one, subnormals of the
    inputs, NaN and infinities, scales at their limits."""
    c = Cache([(16, 16)] * 6, 1, 64, 16, 16, seed=2)
    k = torch.zeros(6, 16, 1, 64)
    k[1] = 448.0
    k[2] = 448.5
    k[2, 3] = -2.0 ** -9
    k[3] = 2.0 ** -24
    k[4, 0, 0, :4] = torch.tensor([float("nan"), float("inf"), -float("inf"), 3.0])
    k[5] = 1.0
    k[5, 1, 0, 0] = 60000.0
    k = k.half()
    codes, scales = [x.clone() for x in c.codes], c.scales.clone()
    bd = torch.zeros(c.n_pages, 1, 1, 2, 64, dtype=torch.uint8)
    want = append_reference(c, k, k, codes, scales, bd)
    assert want == vae4.STATUS_BAD_VALUE
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv, sc, bdd = run_append(c, k, k, "tokens", True, status)
    assert int(status) == want
    # (the bounds of blocks without tokens keep the buffer's own contents)
    used = c.table[:, 0].long()
    assert torch.equal(sc.cpu().nan_to_num(-1), scales.nan_to_num(-1))
    for got, w in zip(kv, codes):
        assert same_values(got.cpu(), w, torch.float8_e4m3fn)
    assert same_values(bdd.cpu()[used], bd[used], torch.float8_e4m3fn)
    s = [float(sc[int(c.table[b, 0]), 0, 0, 0]) for b in range(6)]
    assert s[0] == 2.0 ** -30 and s[1] == 1.0 and s[2] == 2.0
    # BF16 values past every scale saturate and are reported
    c = Cache([(1, 1)], 1, 64, 16, 16, seed=2)
    x = torch.full((1, 1, 1, 64), 1e30).bfloat16()
    status.zero_()
    kv, sc, _ = run_append(c, x, x, "tokens", False, status)
    assert int(status) == vae4.STATUS_BAD_VALUE
    pg = int(c.table[0, 0])
    assert float(sc[pg, 1, 0, 0]) == 2.0 ** 30 and (kv[1][pg, 0] == 0x7E).all()


def test_append_refuses_pages_scales_and_lengths():
    lens = [(20, 2), (20, 2), (20, 2), (20, 2)]
    c = Cache(lens, 1, 64, 16, 16, seed=8)
    c.scales = torch.exp2(c.scales.log2().round())
    c.table[0, 1] = c.n_pages                      # no such page
    c.scales[int(c.table[1, 1]), 0] = float("nan")  # the old scale of K
    c.seq = torch.tensor([[20, 2], [20, 2], [20, 21], [1000, 2]], dtype=torch.int32)
    x = torch.randn(4, 2, 1, 64).half()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv, sc, _ = run_append(c, x, x, "tokens", False, status)
    assert int(status) == (vae4.STATUS_BAD_BLOCK | vae4.STATUS_BAD_SCALE | vae4.STATUS_BAD_QLEN |
                           vae4.STATUS_BAD_LENGTH)
    pg = int(c.table[1, 1])
    want = [x.clone() for x in c.codes]
    got = [x.cpu() for x in kv]
    assert torch.equal(got[0], want[0])            # no K was written anywhere
    want[1][pg] = got[1][pg]                       # the V of sequence 1 was
    assert torch.equal(got[1], want[1])
    assert not torch.equal(got[1][pg], c.codes[1][pg])


# ------------------------------------------------------------------ together
def test_caches_past_32_bit_offsets():
    """Pages, scales and bounds a GB apart: the same bits as when they lie
    together."""
    gb = 1 << 30
    c = Cache([(250, 3), (60, 2)], 2, 128, 64, 32, seed=16, extra=1)
    q, bd = queries(c, 3, 4), bounds_of(c)
    k_new = torch.randn(2, 3, 2, 128, generator=torch.Generator().manual_seed(1)).half()
    assert c.n_pages == 6
    buf = torch.zeros(6 * gb, dtype=torch.uint8, device="cuda")
    near = dict(k=c.codes[0].cuda(), v=c.codes[1].cuda(), sc=c.scales.cuda(), bd=bd.cuda())
    far = dict(k=buf.as_strided((6, 64, 2, 128), (gb, 256, 128, 1)),
               v=buf.as_strided((6, 64, 2, 128), (gb, 256, 128, 1), gb // 4),
               sc=buf.view(torch.float32).as_strided((6, 2, 2, 2), (gb // 4, 4, 2, 1), gb // 8),
               bd=buf.as_strided((6, 2, 2, 2, 128), (gb, 1024, 512, 128, 1), 3 * gb // 4))
    for name, t in near.items():
        far[name].copy_(t)
    qd, bt, seq, kd = dev(q, c.table, c.seq, k_new)
    got = []
    for d in (near, far):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        outs = [torch.zeros_like(qd), torch.zeros_like(qd)]
        scores = torch.zeros(2, 3, 2, 8, device="cuda")
        ids = torch.zeros(2, 3, 2, 4, dtype=torch.int32, device="cuda")
        ws = vae4.alloc_sparse_workspace(2, 8, 2, 3, 128, 64 * c.table.shape[1], 32, 4)
        wd = vae4.alloc_workspace(2, 8, 2, 3, 128, 64 * c.table.shape[1])
        vae4.verify_attn_e4m3_append(kd, kd, d["k"], d["v"], bt, seq, d["sc"], k_bounds=d["bd"], status=status)
        vae4.verify_attn_e4m3_block_scaled(qd, d["k"], d["v"], bt, seq, d["sc"], outs[0], wd)
        vae4.verify_attn_e4m3_block_scores(qd, d["bd"], bt, seq, d["sc"], scores, block_tokens=32, status=status)
        vae4.verify_attn_e4m3_select_blocks(scores, seq, ids, block_tokens=32, local_blocks=1, status=status)
        vae4.verify_attn_e4m3_sparse(qd, d["k"], d["v"], bt, seq, d["sc"], ids, outs[1], ws)
        assert int(status) == 0 and vae4.read_status(ws) == 0 and vae4.read_status(wd) == 0
        assert outs[0].any() and torch.isfinite(outs[0]).all()
        got.append([d["k"], d["v"], d["sc"].contiguous().view(torch.int32), d["bd"], scores, ids] + outs)
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_steps_in_a_row_wait_for_one_another():
    """Twenty steps enqueued without a pause, each kernel's input the one
    before's output, give the bits of the steps run one by one."""
    B, Q, G, H, D, page, blk, k, steps = 3, 4, 4, 2, 128, 64, 16, 6, 20
    g = torch.Generator(device="cuda").manual_seed(17)
    new = [torch.randn(steps, B, Q, H, D, generator=g, device="cuda").half() for _ in (0, 1)]
    q = torch.randn(steps, B, Q, G * H, D, generator=g, device="cuda").half()
    pages = 12
    table = torch.randperm(B * pages, generator=g, device="cuda").int().view(B, pages)
    seqs = [torch.tensor([[Q * (t + 1) + 100 * b, Q] for b in range(B)], dtype=torch.int32, device="cuda")
            for t in range(steps)]
    first = torch.tensor([[100 * b, 100 * b] for b in range(B)], dtype=torch.int32, device="cuda")
    prompt = torch.randn(2, B, 200, H, D, generator=g, device="cuda").half()
    runs = []
    for pause in (True, False):
        kv = torch.zeros(B * pages, 2, H, page, D, dtype=torch.uint8, device="cuda")
        kc, vc = vae4.cache_views(kv)
        sc = vae4.alloc_block_scales(B * pages, H, page, blk)
        bd = vae4.alloc_k_bounds(B * pages, H, page, blk, D)
        scores = torch.zeros(steps, B, Q, H, pages * page // blk, device="cuda")
        ids = torch.zeros(steps, B, Q, H, k, dtype=torch.int32, device="cuda")
        outs = torch.zeros(2, steps, B, Q, G * H, D, dtype=torch.float16, device="cuda")
        ws = vae4.alloc_workspace(B, G * H, H, Q, D, pages * page)
        wl = vae4.alloc_sparse_workspace(B, G * H, H, Q, D, pages * page, blk, k)
        torch.cuda.synchronize()
        wait = torch.cuda.synchronize if pause else (lambda: None)
        vae4.verify_attn_e4m3_append(prompt[0], prompt[1], kc, vc, table, first, sc, k_bounds=bd)
        wait()
        for t in range(steps):
            vae4.verify_attn_e4m3_append(new[0][t], new[1][t], kc, vc, table, seqs[t], sc, k_bounds=bd)
            wait()
            vae4.verify_attn_e4m3_block_scaled(q[t], kc, vc, table, seqs[t], sc, outs[0, t], ws)
            wait()
            vae4.verify_attn_e4m3_block_scores(q[t], bd, table, seqs[t], sc, scores[t], block_tokens=blk)
            wait()
            vae4.verify_attn_e4m3_select_blocks(scores[t], seqs[t], ids[t], block_tokens=blk)
            wait()
            vae4.verify_attn_e4m3_sparse(q[t], kc, vc, table, seqs[t], sc, ids[t], outs[1, t], wl)
            wait()
        torch.cuda.synchronize()
        assert vae4.read_status(ws) == 0 and vae4.read_status(wl) == 0
        assert outs[0].any() and outs[1].any() and torch.isfinite(outs).all()
        runs.append((kv, sc.view(torch.int32), bd, scores.view(torch.int32), ids, outs))
    for a, b in zip(*runs):
        assert torch.equal(a, b)


def test_captured_calls_on_two_branches():
    """A graph whose branches run side by side after the writer and join before
    the sparse call gives the bits of the calls one by one, on every replay."""
    c = Cache([(3000, 3), (700, 2)], 2, 128, 64, 16, seed=18)
    Q, G, k = 3, 4, 9
    q, bd = queries(c, Q, G), bounds_of(c)
    x = torch.randn(2, Q, 2, 128, generator=torch.Generator().manual_seed(3)).half()
    cap = c.table.shape[1] * c.page
    qd, bt, seq, xd = dev(q, c.table, c.seq, x)
    kv0, sc0, bd0 = c.device(), c.scales.cuda(), bd.cuda()
    kc, vc, sc, bdd = kv0[0].clone(), kv0[1].clone(), sc0.clone(), bd0.clone()
    scores = torch.zeros(2, Q, 2, cap // 16, device="cuda")
    ids = torch.zeros(2, Q, 2, k, dtype=torch.int32, device="cuda")
    outs = torch.zeros(2, *qd.shape, dtype=torch.float16, device="cuda")
    ws = vae4.alloc_workspace(2, 8, 2, Q, 128, cap)
    wl = vae4.alloc_sparse_workspace(2, 8, 2, Q, 128, cap, 16, k)

    def step(main, side):
        wait = torch.cuda.synchronize if side is None else (lambda: None)
        vae4.verify_attn_e4m3_append(xd, xd, kc, vc, bt, seq, sc, k_bounds=bdd)
        wait()
        if side is not None:
            side.wait_stream(main)
        vae4.verify_attn_e4m3_block_scores(qd, bdd, bt, seq, sc, scores, block_tokens=16, stream=side)
        wait()
        vae4.verify_attn_e4m3_select_blocks(scores, seq, ids, block_tokens=16, stream=side)
        wait()
        vae4.verify_attn_e4m3_block_scaled(qd, kc, vc, bt, seq, sc, outs[0], ws)
        wait()
        if side is not None:
            main.wait_stream(side)
        vae4.verify_attn_e4m3_sparse(qd, kc, vc, bt, seq, sc, ids, outs[1], wl)
        wait()

    def restore():
        for t, o in ((kc, kv0[0]), (vc, kv0[1]), (sc, sc0), (bdd, bd0)):
            t.copy_(o)
        for t in (scores, ids, outs):
            t.zero_()
        torch.cuda.synchronize()

    step(None, None)
    want = [t.clone() for t in (kc, vc, sc, bdd, scores, ids, outs)]
    restore()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(torch.cuda.current_stream(), side)
    for _ in range(5):
        restore()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip((kc, vc, sc, bdd, scores, ids, outs), want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert vae4.read_status(ws) == 0 and vae4.read_status(wl) == 0


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_decoding_steps_together(graph, fmt):
    """Prompt, then steps of drafts of which some are rejected: append, scores,
    choice, sparse and whole attention, eager or as one captured graph whose
    lengths change from replay to replay, on a stream of its own.  After each
    step the outputs are those of the definitions on the cache's contents."""
    B, Q, Hkv, G, D, page, blk, k = 3, 4, 2, 3, 128, 64, 32, 5
    flags = FMT[fmt][2]
    cap = 640
    c = Cache([(cap, Q)] * B, Hkv, D, page, blk, fmt, seed=11)
    g = torch.Generator().manual_seed(5)
    kc, vc = [torch.full_like(x, 0x7F).cuda() for x in c.codes]
    bt = c.table.cuda()
    sc = vae4.alloc_block_scales(c.n_pages, Hkv, page, blk)
    bd = vae4.alloc_k_bounds(c.n_pages, Hkv, page, blk, D)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    prompts = [200, 333, 64]
    new = torch.randn(2, B, 333, Hkv, D, generator=g).half().cuda()
    seq = torch.tensor([(n, n) for n in prompts], dtype=torch.int32, device="cuda")
    vae4.verify_attn_e4m3_append(new[0], new[1], kc, vc, bt, seq, sc, k_bounds=bd, status=status,
                                 flags=flags)
    q = torch.zeros(B, Q, G * Hkv, D, dtype=torch.float16, device="cuda")
    kn, vn = [torch.zeros(B, Q, Hkv, D, dtype=torch.float16, device="cuda") for _ in range(2)]
    out, whole = torch.empty_like(q), torch.empty_like(q)
    scores = torch.zeros(B, Q, Hkv, cap // blk, device="cuda")
    ids = torch.zeros(B, Q, Hkv, k, dtype=torch.int32, device="cuda")
    ws = vae4.alloc_sparse_workspace(B, G * Hkv, Hkv, Q, D, cap, blk, k)
    ws2 = vae4.alloc_workspace(B, G * Hkv, Hkv, Q, D, cap)

    def step():
        vae4.verify_attn_e4m3_append(kn, vn, kc, vc, bt, seq, sc, k_bounds=bd, status=status, flags=flags)
        vae4.verify_attn_e4m3_block_scores(q, bd, bt, seq, sc, scores, block_tokens=blk, status=status,
                                           flags=flags)
        vae4.verify_attn_e4m3_select_blocks(scores, seq, ids, block_tokens=blk, sink_blocks=1,
                                            local_blocks=1, status=status)
        vae4.verify_attn_e4m3_sparse(q, kc, vc, bt, seq, sc, ids, out, ws, max_seq_len=cap, flags=flags)
        vae4.verify_attn_e4m3_block_scaled(q, kc, vc, bt, seq, sc, whole, ws2, max_seq_len=cap, flags=flags)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    captured = None
    lens = prompts
    with torch.cuda.stream(stream):
        if graph:
            captured = torch.cuda.CUDAGraph()
            with torch.cuda.graph(captured, stream=stream):
                step()
        for it in range(4):
            drafts = [(4, 1, 3), (2, 4, 4), (1, 1, 1), (3, 0, 4)][it]
            pairs = [(L + n if n else 0, n) for L, n in zip(lens, drafts)]
            q.copy_(torch.randn(q.shape, generator=g))
            kn.copy_(torch.randn(kn.shape, generator=g) * 2.0 ** (it - 1))
            vn.copy_(torch.randn(vn.shape, generator=g) * 2.0 ** (1 - it))
            seq.copy_(torch.tensor(pairs, dtype=torch.int32))
            captured.replay() if graph else step()
            stream.synchronize()
            assert int(status) == 0 and vae4.read_status(ws) == 0 and vae4.read_status(ws2) == 0
            now = Cache(pairs, Hkv, D, page, blk, fmt, seed=1)
            now.table, now.n_pages = c.table, c.n_pages
            now.codes, now.scales = [kc.cpu(), vc.cpu()], sc.cpu()
            idc, sco = ids.cpu(), scores.cpu()
            for b, (L, n) in enumerate(pairs):
                for i in range(Q):
                    v = (L - n + i) // blk + 1 if L and i < n else 0
                    for h in range(Hkv):
                        assert idc[b, i, h].tolist() == choose(sco[b, i, h].tolist(), v, k, 1, 1)
            check(out.cpu(), *reference(now, q.cpu(), allowed=listed(now, idc)))
            check(whole.cpu(), *reference(now, q.cpu()))
            # the last draft of a sequence that had several is rejected
            lens = [L - (n > 1) if n else M for (L, n), M in zip(pairs, lens)]
    torch.cuda.current_stream().wait_stream(stream)
