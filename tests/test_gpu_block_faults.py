"""The block-scaled cache's calls where they can go wrong: waits that run out,
host threads at once, weights far below the largest, NaN queries, invalid
scales.  References and their tolerances as in test_gpu_blocks.py, unless a
test derives its own."""
import math
import threading
import threading

import pytest
import torch

import fp8_paged_attention_e4m3_gb300 as vae4
from test_gpu_blocks import FMT, Cache, bounds_of, check, dev, listed, queries, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    vae4.load()


def guarded(shape, fill):
    """An FP16 tensor within a larger buffer, and the buffer's other elements."""
    n, pad = math.prod(shape), 4096
    buf = torch.full((n + 2 * pad,), fill, dtype=torch.float16, device="cuda")
    return buf[pad:pad + n].view(shape), (buf[:pad], buf[pad + n:])


TIMEOUTS = [
    # lens, Q, G, Hkv, D, page, block, layout, num_sms
    ([(3000, 4), (100, 4), (50, 2)], 4, 3, 2, 128, 32, 16, "tokens", 0),
    ([(2000, 8)], 8, 6, 1, 256, 16, 16, "tokens", 0),
    ([(700, 16), (90, 16)], 16, 6, 2, 64, 32, 32, "pool", 5),      # two row groups
    ([(300, 2)] * 5, 2, 2, 2, 128, 32, 16, "padded", 0),           # 8-byte copies
    ([(130 + b, 1) for b in range(30)], 1, 2, 4, 64, 16, 16, "tokens", 1),  # 120 segments of one CTA
]


def timed_out(c, q, layout, num_sms, repeats):
    """Calls whose waits all run out, `repeats` dense and as many sparse ones,
    and after them one of each that is left alone."""
    Q, Hq = q.shape[1:3]
    k, v = c.device(layout)
    qd, bt, seq, sc = dev(q, c.table, c.seq, c.scales)
    B, cap = len(c.lens), c.table.shape[1] * c.page
    ids = torch.arange(5, dtype=torch.int32).expand(B, Q, c.Hkv, 5).contiguous()
    idd = ids.cuda()
    for sp in (False, True):
        n = (vae4.sparse_workspace_bytes(B, Hq, c.Hkv, Q, c.D, cap, c.blk, 5, num_sms) if sp else
             vae4.block_scaled_workspace_bytes(B, Hq, c.Hkv, Q, c.D, cap, num_sms))
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        for it in range(repeats + 1):
            flags = vae4.FLAG_TEST_SHORT_WAITS if it < repeats else 0
            out, guards = guarded(q.shape, 3.0)
            if sp:
                vae4.verify_attn_e4m3_sparse(qd, k, v, bt, seq, sc, idd, out, ws, flags=flags,
                                             num_sms=num_sms)
            else:
                vae4.verify_attn_e4m3_block_scaled(qd, k, v, bt, seq, sc, out, ws, flags=flags,
                                                   num_sms=num_sms)
            torch.cuda.synchronize()
            assert all((g == 3).all() for g in guards)
            assert vae4.read_status(ws) == (vae4.STATUS_TIMEOUT if flags else 0)
            if flags:
                assert not out.any()
                vae4.clear_status(ws)
        check(out.cpu(), *reference(c, q, allowed=listed(c, ids) if sp else None))


@pytest.mark.parametrize("lens,Q,G,Hkv,D,page,blk,layout,num_sms", TIMEOUTS)
def test_waits_that_run_out_end_the_call_every_time(lens, Q, G, Hkv, D, page, blk, layout, num_sms):
    """Whichever role gives up first, and however late the others look: the
    call ends, its rows are zero, and nothing past them is written."""
    c = Cache(lens, Hkv, D, page, blk, seed=31)
    timed_out(c, queries(c, Q, G), layout, num_sms, 40)


@pytest.mark.parametrize("lens,Q,G,Hkv,D,page,blk,layout,num_sms", [
    ([(130 + 7 * b, 1) for b in range(40)], 1, 2, 4, 64, 16, 16, "tokens", 1),
    ([(200 + b, 3) for b in range(70)], 3, 4, 2, 128, 64, 32, "padded", 2),
    ([(90, 2)] * 50, 2, 1, 3, 256, 32, 16, "pool", 1),
])
def test_waits_that_run_out_with_segments_left(lens, Q, G, Hkv, D, page, blk, layout, num_sms):
    """More than 32 groups and more segments a CTA than it plans at a time: the
    later ones are planned while copies of the first may be in flight."""
    c = Cache(lens, Hkv, D, page, blk, seed=32)
    assert len(lens) * Hkv > 64 * num_sms
    timed_out(c, queries(c, Q, G), layout, num_sms, 20)


def test_sparse_calls_of_two_host_threads():
    """Two host threads whose visit lists need different amounts of shared
    memory, both above the default limit, on a stream each: every call is
    launched, and each gives what it gives alone."""
    q = torch.randn(1, 2, 4, 64, generator=torch.Generator().manual_seed(3)).half()
    work = []
    for blocks in (24600, 98304):
        c = Cache([(500, 2)], 1, 64, 16, 16, seed=33)
        table = torch.full((1, blocks), -1, dtype=torch.int32)
        table[:, :c.table.shape[1]] = c.table
        ids = torch.tensor([0, 3, 17, 31], dtype=torch.int32).expand(1, 2, 1, 4).contiguous()
        k, v = c.device()
        qd, bt, seq, sc, idd = dev(q, table, c.seq, c.scales, ids)
        ws = vae4.alloc_sparse_workspace(1, 4, 1, 2, 64, blocks * 16, 16, 4)
        work.append((c, ids, (qd, k, v, bt, seq, sc, idd, torch.zeros_like(qd), ws), torch.cuda.Stream()))
    torch.cuda.synchronize()
    go, errors = threading.Barrier(len(work)), []

    def calls(args, stream):
        try:
            go.wait()
            for _ in range(3000):
                vae4.verify_attn_e4m3_sparse(*args, stream=stream)
        except Exception as e:  # reported by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=calls, args=w[2:]) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for c, ids, args, _ in work:
        assert vae4.read_status(args[-1]) == 0
        check(args[-2].cpu(), *reference(c, q, allowed=listed(c, ids)))


@pytest.mark.parametrize("L,sparse_call", [(64, False), (3000, False), (64, True), (3000, True)])
@pytest.mark.parametrize("far", [6, 13, 20, 26])
def test_small_scales_beside_a_large_one_with_zero_codes(L, sparse_call, far):
    """One block's s_V is 2^far times the others', its codes are zero in half of
    the channels: what the other blocks give there is seen to the stated bound.
    With p = e^z / sum e^z, w = p s_V, W its largest in the row and c the codes:
        |got - out| <= (2^-11 + 2^-11) sum w |c| + 2^-25 W sum |c| + 2^-11 |out| + 2^-25
    (weights: 2^-11 and 2^-25 W; as much again for FP32 scores and sums, which are
    off by less; out rounded to FP16)."""
    c = Cache([(L, 2)], 1, 64, 16, 16, seed=34)
    q = queries(c, 2, 3)
    n_blk = -(-L // 16)
    c.scales[:, 1] = torch.where(c.scales[:, 1].isnan(), c.scales[:, 1], torch.tensor(1.0))
    big = int(c.table[0, 1])
    c.scales[big, 1] = 2.0 ** far
    c.codes[1][big, :, :, :32] = 0
    if far > 7:  # the other channels inside FP16's range
        c.codes[1][big, :, :, 32:] &= 0x83
    K, s = c.values(0, 0), c.scales[c.table[0, :n_blk].long(), 1, 0, 0].double().repeat_interleave(16)[:L]
    codes = c.values(1, 0)[:, 0] / s[:, None]
    ids = torch.arange(n_blk, dtype=torch.int32).expand(1, 2, 1, n_blk).contiguous()
    k, v = c.device()
    qd, bt, seq, sc, idd = dev(q, c.table, c.seq, c.scales, ids)
    out, cap = torch.zeros_like(qd), c.table.shape[1] * 16
    if sparse_call:
        ws = vae4.alloc_sparse_workspace(1, 3, 1, 2, 64, cap, 16, n_blk)
        vae4.verify_attn_e4m3_sparse(qd, k, v, bt, seq, sc, idd, out, ws)
    else:
        ws = vae4.alloc_workspace(1, 3, 1, 2, 64, cap)
        vae4.verify_attn_e4m3_block_scaled(qd, k, v, bt, seq, sc, out, ws)
    assert vae4.read_status(ws) == 0
    for i in range(2):
        z = q[0, i].double() @ K[:L - 1 + i, 0].T / 8
        p = torch.softmax(z, -1)
        w, cc = p * s[:L - 1 + i], codes[:L - 1 + i]
        ref = w @ cc
        tol = (2.0 ** -10 * (w @ cc.abs()) + 2.0 ** -25 * w.amax(-1, keepdim=True) * cc.abs().sum(0) +
               2.0 ** -11 * ref.abs() + 2.0 ** -25)
        assert ref.abs().max() < 6e4
        far_off = ((out[0, i].cpu().double() - ref).abs() - tol).max().item()
        assert far_off <= 0, far_off


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("lens,Q,G,Hkv,D,num_sms", [
    ([(300, 3), (90, 2)], 3, 4, 2, 128, 1),                    # units finished by their CTA
    ([(5000, 3)], 3, 4, 2, 64, 0),                             # a part per SM, combined by rows
    ([(4000, 3)] + [(1500, 2)] * 5, 3, 2, 2, 128, 0),          # combined by warps
    ([(2000, 16)], 16, 6, 1, 256, 0),                          # two row groups
])
def test_a_query_with_a_nan_gives_a_row_of_nan(lens, Q, G, Hkv, D, num_sms, value):
    """And all others keep their values; in the dense and in the sparse form."""
    c = Cache(lens, Hkv, D, 32, 16, seed=35)
    q = queries(c, Q, G)
    odd = [(0, 0, 0), (0, Q - 1, G * Hkv - 1), (len(lens) - 1, 1, G)] if Hkv > 1 else [(0, 0, 0), (0, 15, 5)]
    for k, (b, i, h) in enumerate(odd):
        q[b, i, h, 7 + 20 * k] = value
    n_blk = -(-max(L for L, _ in lens) // 16)
    ids = torch.arange(n_blk, dtype=torch.int32).expand(len(lens), Q, Hkv, n_blk).contiguous()
    k, v = c.device()
    qd, bt, seq, sc, idd = dev(q, c.table, c.seq, c.scales, ids)
    clean = q.clone()
    for b, i, h in odd:
        clean[b, i, h] = 0
    ref, tol = reference(c, clean)
    cap, B, Hq = c.table.shape[1] * 32, len(lens), G * Hkv
    for sp in (False, True):
        out = torch.zeros_like(qd)
        n = (vae4.sparse_workspace_bytes(B, Hq, Hkv, Q, D, cap, 16, n_blk, num_sms) if sp else
             vae4.block_scaled_workspace_bytes(B, Hq, Hkv, Q, D, cap, num_sms))
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        if sp:
            vae4.verify_attn_e4m3_sparse(qd, k, v, bt, seq, sc, idd, out, ws, num_sms=num_sms)
        else:
            vae4.verify_attn_e4m3_block_scaled(qd, k, v, bt, seq, sc, out, ws, num_sms=num_sms)
        assert vae4.read_status(ws) == 0
        got = out.cpu()
        for b, i, h in odd:
            assert got[b, i, h].isnan().all(), (sp, b, i, h)
            got[b, i, h] = ref[b, i, h].half()
        check(got, ref, tol)


@pytest.mark.parametrize("Q,G,head", [(1, 4, 0), (3, 6, 5), (8, 12, 3), (2, 1, 0)])
def test_scores_of_a_query_with_a_nan_are_nan(Q, G, head):
    """In whichever head of the group it is; other queries and KV heads keep
    their scores, and blocks that the query does not see score -inf."""
    c = Cache([(400, Q), (50, 1)], 2, 64, 32, 16, seed=36)
    q, bd = queries(c, Q, G), bounds_of(c)
    qd, bdd, bt, seq, sc = dev(q, bd, c.table, c.seq, c.scales)
    scores = torch.full((2, 2, Q, 2, 25), 5.0, device="cuda")
    vae4.verify_attn_e4m3_block_scores(qd, bdd, bt, seq, sc, scores[0], block_tokens=16)
    qd[0, Q - 1, G + head, 9] = float("nan")
    vae4.verify_attn_e4m3_block_scores(qd, bdd, bt, seq, sc, scores[1], block_tokens=16)
    clean, got = scores.cpu()
    seen = (400 - 1) // 16 + 1
    assert got[0, Q - 1, 1, :seen].isnan().all()
    got[0, Q - 1, 1, :seen] = clean[0, Q - 1, 1, :seen]
    assert torch.equal(got, clean)


@pytest.mark.parametrize("bad", [0.0, -1.0, float("nan"), float("inf"), 2.0 ** 41, 2.0 ** -41])
def test_scores_report_invalid_scales(bad):
    """A K scale outside 2^-40 .. 2^40: -inf for its block and head, and the
    status bit; the limits themselves, V's scales and those of blocks without
    tokens do no harm."""
    c = Cache([(230, 2), (40, 1)], 2, 64, 32, 16, seed=37)
    q, bd = queries(c, 2, 3), bounds_of(c)
    qd, bdd, bt, seq, sc = dev(q, bd, c.table, c.seq, c.scales)
    sc[int(c.table[0, 2]), 0, 0, 0], sc[int(c.table[0, 3]), 0, 0, 0] = 2.0 ** 40, 2.0 ** -40
    sc[int(c.table[0, 4]), 1] = bad
    scores = torch.full((2, 2, 2, 2, 15), 5.0, device="cuda")
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    vae4.verify_attn_e4m3_block_scores(qd, bdd, bt, seq, sc, scores[0], block_tokens=16, status=status[:1])
    sc[int(c.table[0, 1]), 0, 1, 1] = bad  # block 3 of head 1
    vae4.verify_attn_e4m3_block_scores(qd, bdd, bt, seq, sc, scores[1], block_tokens=16, status=status[1:])
    clean, got = scores.cpu()
    assert status.tolist() == [0, vae4.STATUS_BAD_SCALE]
    assert (got[0, :, 1, 3] == -math.inf).all() and clean[0, :, 1, 3].isfinite().all()
    got[0, :, 1, 3] = clean[0, :, 1, 3]
    assert torch.equal(got, clean)


def one_token(B, H, G, D, seed):
    """Sequences of one token each: whatever the scores, a row is its V."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    table = torch.randperm(B, generator=g, device="cuda").int().view(B, 1)
    x = torch.randn(2, B, 1, H, D, generator=g, device="cuda").half()
    q = torch.randn(B, 1, G * H, D, generator=g, device="cuda").half()
    cache = [torch.full((B, 16, H, D), 0x7F, dtype=torch.uint8, device="cuda") for _ in (0, 1)]
    return (table, x, q, cache, vae4.alloc_block_scales(B, H, 16, 16),
            vae4.alloc_k_bounds(B, H, 16, 16, D), torch.ones(B, 2, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("B,H,G", [(65535, 1, 1), (1, 32767, 2), (300, 200, 1), (2, 1, 96), (1, 3, 32)])
def test_the_largest_grids(B, H, G):
    """The most sequences and KV heads that the calls take, and the most heads
    on one KV head: append, attention, scores, choice and sparse attention."""
    D = 64
    table, x, q, (kc, vc), sc, bd, seq = one_token(B, H, G, D, B + H)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    vae4.verify_attn_e4m3_append(x[0], x[1], kc, vc, table, seq, sc, k_bounds=bd, status=status)
    pg = table[:, 0].long()
    v = vc[pg, 0].view(torch.float8_e4m3fn).float() * sc[pg, 1, :, :1]        # [B][H][D]
    k = kc[pg, 0].view(torch.float8_e4m3fn).float() * sc[pg, 0, :, :1]
    for got, new in ((k, x[0]), (v, x[1])):  # a code is off by at most half a step: 2^-4, or 2^-10 s
        new = new[:, 0].float()
        assert ((got - new).abs() <= 2.0 ** -4 * new.abs() + 2.0 ** -10 * new.abs().amax(-1, keepdim=True) / 224).all()
    want = v.half().repeat_interleave(G, 1)[:, None]
    out, out2 = torch.zeros_like(q), torch.zeros_like(q)
    scores = torch.zeros(B, 1, H, 1, device="cuda")
    ids = torch.full((B, 1, H, 2), 7, dtype=torch.int32, device="cuda")
    ws = vae4.alloc_workspace(B, G * H, H, 1, D, 16)
    wl = vae4.alloc_sparse_workspace(B, G * H, H, 1, D, 16, 16, 2)
    vae4.verify_attn_e4m3_block_scaled(q, kc, vc, table, seq, sc, out, ws)
    vae4.verify_attn_e4m3_block_scores(q, bd, table, seq, sc, scores, block_tokens=16, status=status)
    vae4.verify_attn_e4m3_select_blocks(scores, seq, ids, block_tokens=16, status=status)
    vae4.verify_attn_e4m3_sparse(q, kc, vc, table, seq, sc, ids, out2, wl)
    assert int(status) == 0 and vae4.read_status(ws) == 0 and vae4.read_status(wl) == 0
    for o in (out, out2):  # one weight of 1 and one division: the rounding to FP16, and 2^-11 for the rest
        assert ((o.float() - want.float()).abs() <= 2.0 ** -10 * want.float().abs() + 2.0 ** -24).all()
    assert (ids[..., 0] == 0).all() and (ids[..., 1] == -1).all()
    z = torch.einsum("bhgd,bhd->bhg", q[:, 0].double().view(B, H, G, D), k.double()).amax(-1) / 8
    mags = torch.einsum("bhgd,bhd->bhg", q[:, 0].double().abs().view(B, H, G, D), k.double().abs()).amax(-1) / 8
    assert ((scores[:, 0, :, 0].double() - z).abs() <= (2 * D + 4) * 2.0 ** -24 * mags).all()


def test_lengths_without_q_and_strided_arguments():
    """[B] lengths (q = Qmax for all) and rows that do not lie together: every
    argument a view into a larger tensor, whose other elements stay as they are."""
    B, Q, H, G, D, page, blk, cap = 3, 3, 2, 4, 128, 64, 16, 256
    lens = [(150, Q), (3, Q), (77, Q)]
    c = Cache(lens, H, D, page, blk, seed=38)
    c.scales = torch.exp2(c.scales.log2().round())  # as earlier calls left them
    g = torch.Generator().manual_seed(4)
    q = queries(c, Q, G)
    x = torch.randn(2, B, Q, H, D, generator=g).half()

    def wide(t, extra):
        big = torch.full([n + e for n, e in zip(t.shape, extra)], 9, dtype=t.dtype, device="cuda")
        view = big[tuple(slice(0, n) for n in t.shape)]
        view.copy_(t)
        return big, view

    results = []
    for strided in (False, True):
        e = (lambda *n: n) if strided else (lambda *n: [0] * len(n))
        kc, vc = c.device()
        seq = wide(torch.tensor(lens, dtype=torch.int32), (0, 1))[1][:, 0] if strided else c.seq[:, 0].contiguous().cuda()
        table = wide(c.table, e(0, 3))[1]
        sc = wide(c.scales, e(0, 1, 1, 0))[1]
        bd = wide(bounds_of(c), e(0, 1, 0, 0, 0))[1]
        qd, xk, xv = wide(q, e(1, 1, 1, 8))[1], wide(x[0], e(0, 2, 1, 16))[1], wide(x[1], e(1, 0, 3, 8))[1]
        cols = cap // blk
        sbig, scores = wide(torch.zeros(B, Q, H, cols), e(0, 1, 1, 5))
        ibig, ids = wide(torch.zeros(B, Q, H, 4, dtype=torch.int32), e(1, 1, 1, 3))
        obig, out = wide(torch.zeros_like(q), e(0, 1, 2, 8))
        o2big, out2 = wide(torch.zeros_like(q), e(0, 0, 1, 8))
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        top = table.shape[1] * page
        ws, wl = vae4.alloc_workspace(B, G * H, H, Q, D, top), vae4.alloc_sparse_workspace(B, G * H, H, Q, D, top, blk, 4)
        vae4.verify_attn_e4m3_append(xk, xv, kc, vc, table, seq, sc, k_bounds=bd, status=status)
        vae4.verify_attn_e4m3_block_scaled(qd, kc, vc, table, seq, sc, out, ws)
        vae4.verify_attn_e4m3_block_scores(qd, bd, table, seq, sc, scores, block_tokens=blk, status=status)
        vae4.verify_attn_e4m3_select_blocks(scores, seq, ids, block_tokens=blk, status=status)
        vae4.verify_attn_e4m3_sparse(qd, kc, vc, table, seq, sc, ids, out2, wl)
        assert int(status) == 0 and vae4.read_status(ws) == 0 and vae4.read_status(wl) == 0
        results.append([kc, vc, sc.contiguous().view(torch.int32), bd, scores, ids, out, out2])
        for big, view in ((sbig, scores), (ibig, ids), (obig, out), (o2big, out2)):
            rest = big.clone()
            rest[tuple(slice(0, n) for n in view.shape)] = 9
            assert (rest == 9).all()
    for a, b in zip(*results):
        assert torch.equal(a, b)
    now = Cache(lens, H, D, page, blk, seed=38)
    now.table, now.codes = c.table, [results[0][0].cpu(), results[0][1].cpu()]
    now.scales = results[0][2].view(torch.float32).cpu()
    check(results[0][6].cpu(), *reference(now, q))
    check(results[0][7].cpu(), *reference(now, q, allowed=listed(now, results[0][5].cpu())))


def test_a_query_whose_scores_are_all_minus_infinity_gives_zeros():
    """An infinite query against keys that are all negative in its channel."""
    c = Cache([(900, 2)], 1, 64, 16, 16, seed=39)
    c.codes[0][..., 3] = torch.where(c.codes[0][..., 3] == 0x7F, c.codes[0][..., 3], torch.tensor(0xB8, dtype=torch.uint8))
    q = queries(c, 2, 3)
    ref, tol = reference(c, q)
    q[0, 1, 2, 3] = float("inf")
    ref[0, 1, 2] = tol[0, 1, 2] = 0
    k, v = c.device()
    qd, bt, seq, sc = dev(q, c.table, c.seq, c.scales)
    out, cap = torch.full_like(qd, 3), c.table.shape[1] * 16
    ws = vae4.alloc_workspace(1, 3, 1, 2, 64, cap)
    vae4.verify_attn_e4m3_block_scaled(qd, k, v, bt, seq, sc, out, ws)
    assert vae4.read_status(ws) == 0
    check(out.cpu(), ref, tol)
