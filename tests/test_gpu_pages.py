"""The pages' entry points on the GPU against plain loops over the definitions.
All results are whole numbers or copied bytes: they have to be equal."""
import random

import pytest
import torch

import fp8_paged_attention_e4m3_gb300 as vae4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    vae4.load()


# ---------------------------------------------------------------------------- plain loops


def count(counts, e, by):
    """The status bits of one entry of page e more or less."""
    if counts[e] == 0:
        return vae4.STATUS_BAD_COUNT
    if counts[e] > 0:
        counts[e] += by
    return 0


def is_page(e, counts):
    return 0 <= e < len(counts)


def odd(e, counts):
    return vae4.STATUS_BAD_BLOCK if e < -1 or e >= len(counts) else 0


def plain_fork(table, counts, parents):
    st, B = 0, len(table)
    par = [p if -1 <= p < B else b for b, p in enumerate(parents)]
    if par != parents:
        st |= vae4.STATUS_BAD_PARENT
    new = [list(table[p]) if p >= 0 else [-1] * len(table[b]) for b, p in enumerate(par)]
    for r, row in enumerate(table):
        more = par.count(r) - 1
        for e in row:
            st |= odd(e, counts)
            if more and is_page(e, counts):
                st |= count(counts, e, more)
    return new, counts, st


def plain_resize(table, counts, seq, page):
    st, cols = 0, len(table[0])
    copies = [[-1, -1] for _ in table]
    ok = []
    for b, (L, q) in enumerate(seq):
        good = 0 <= L <= cols * page and 0 <= q <= L
        if not good:
            st |= vae4.STATUS_BAD_LENGTH if L < 0 or L > cols * page else vae4.STATUS_BAD_QLEN
        ok.append(good)
        for j, e in enumerate(table[b]):
            st |= odd(e, counts)
            if good and j * page >= L and is_page(e, counts):
                table[b][j] = -1
                st |= count(counts, e, -1)
    held = list(counts)
    free = [x for x, c in enumerate(counts) if c == 0]
    for b, (L, q) in enumerate(seq):
        for j in range(cols):
            e = table[b][j]
            if not ok[b] or j * page >= L:
                continue
            mine = e != -1 and not (is_page(e, counts) and (held[e] > 1 or held[e] < 0) and q > 0 and
                                    j >= (L - q) // page)
            if mine:
                continue
            if not free:
                st |= vae4.STATUS_NO_PAGES
                continue
            x = free.pop(0)
            table[b][j], counts[x] = x, 1
            if e >= 0:
                st |= count(counts, e, -1)
                if j == (L - q) // page and (L - q) % page:
                    copies[b] = [e, x]
    return table, counts, copies, st


def plain_compact(table, counts, m):
    st = 0
    n = sum(c != 0 for c in counts)
    holes = [x for x in range(n) if counts[x] == 0]
    movers = [x for x in reversed(range(n, len(counts))) if counts[x] > 0]
    moves = list(zip(movers, holes))[:m]
    to = dict(moves)
    for row in table:
        for j, e in enumerate(row):
            if moves:
                st |= odd(e, counts)
            row[j] = to.get(e, e)
    for a, b in moves:
        counts[b], counts[a] = counts[a], 0
    return table, counts, [list(x) for x in moves] + [[-1, -1]] * (m - len(moves)), st


# ---------------------------------------------------------------------------- pools


def pool(seed, B, cols, extra=9, share=0.5, kept=2, gaps=False):
    """(table, counts): rows of random numbers of pages; some share the start of
    an earlier row, some pages are kept."""
    r = random.Random(seed)
    table, used = [], 0
    for b in range(B):
        n = r.randrange(cols + 1)
        row = [-1] * cols
        s = 0
        if b and r.random() < share:
            lead = table[r.randrange(b)]
            s = r.randrange(min(n, sum(e >= 0 for e in lead)) + 1)
            row[:s] = lead[:s]
        for j in range(s, n):
            row[j] = used
            used += 1
        if gaps and n > 2:
            row[r.randrange(n)] = -1
        table.append(row)
    n_pages = used + extra + kept
    order = list(range(n_pages))
    r.shuffle(order)
    table = [[order[e] if e >= 0 else -1 for e in row] for row in table]
    counts = [0] * n_pages
    for row in table:
        for e in row:
            if e >= 0:
                counts[e] += 1
    for x in order[used:used + kept]:
        counts[x] = -1 - r.randrange(3)
    if kept and used and table[0][0] >= 0:
        counts[table[0][0]] = -5  # a kept page that rows hold
    return table, counts


def dev(x, pad=0):
    t = torch.tensor(x, dtype=torch.int32)
    if pad:  # rows with memory between them
        wide = torch.full((t.shape[0], t.shape[1] + pad), 77, dtype=torch.int32, device="cuda")
        wide[:, :t.shape[1]] = t.cuda()
        return wide[:, :t.shape[1]]
    return t.cuda()


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def lengths(seed, table, page):
    """(L, q) of a next step for each row: grow, shrink, end, begin."""
    r = random.Random(seed)
    out = []
    for row in table:
        had = sum(e >= 0 for e in row)
        kind = r.randrange(5)
        top = len(row) * page
        L = max(0, had * page - r.randrange(page)) if had else 0
        if kind == 0:
            out.append((0, 0))
        elif kind == 1:
            L = r.randrange(L + 1)
            out.append((L, min(L, 1)))
        elif kind == 2:
            out.append((top, r.randrange(top + 1)))
        else:
            q = r.choice([0, 1, 8, page, 2 * page + 3])
            L = min(top, L + q)
            out.append((L, min(q, L)))
    return out


SHAPES = [(1, 1), (1, 7), (3, 1), (5, 33), (8, 64), (31, 100), (257, 65), (2, 5000), (700, 9), (64, 1031)]


@pytest.mark.parametrize("B,cols", SHAPES)
@pytest.mark.parametrize("pad", [0, 3])
def test_fork(B, cols, pad):
    table, counts = pool(B + cols, B, cols)
    r = random.Random(cols)
    parents = [r.choice([b, b, -1, r.randrange(B), r.randrange(B)]) for b in range(B)]
    t, c, st = dev(table, pad), dev(counts), status()
    vae4.verify_attn_e4m3_fork_pages(t, c, dev(parents), status=st)
    want, wc, ws = plain_fork([list(x) for x in table], list(counts), parents)
    assert t.tolist() == want and c.tolist() == wc and int(st) == ws == 0
    if pad and B > 1:
        assert bool((t.as_strided((B, pad), t.stride(), t.storage_offset() + cols) == 77).all())


def test_fork_of_many_rows():
    B = 8192
    table, counts = pool(3, B, 3)
    parents = [(b * 5 + 1) % B if b % 7 else -1 for b in range(B)]
    t, c = dev(table), dev(counts)
    vae4.verify_attn_e4m3_fork_pages(t, c, dev(parents))
    want, wc, _ = plain_fork(table, counts, parents)
    assert t.tolist() == want and c.tolist() == wc


def test_fork_reports():
    table, counts = pool(5, 4, 6, share=0)
    table[1][0], table[2][1] = -9, len(counts)
    table[3][0] = counts.index(0)  # a page that nothing counts
    parents = [1, 4, -2, 0]
    t, c, st = dev(table), dev(counts), status()
    vae4.verify_attn_e4m3_fork_pages(t, c, dev(parents), status=st)
    want, wc, ws = plain_fork([list(x) for x in table], list(counts), parents)
    assert t.tolist() == want and c.tolist() == wc and int(st) == ws
    assert ws == vae4.STATUS_BAD_BLOCK | vae4.STATUS_BAD_PARENT | vae4.STATUS_BAD_COUNT


@pytest.mark.parametrize("B,cols", SHAPES)
@pytest.mark.parametrize("page,gaps", [(16, False), (48, True)])
def test_resize(B, cols, page, gaps):
    table, counts = pool(2 * B + cols, B, cols, extra=B * cols, gaps=gaps)
    seq = lengths(B, table, page)
    t, c, st = dev(table, 3 if gaps else 0), dev(counts), status()
    copies = torch.full((B, 2), 55, dtype=torch.int32, device="cuda")
    ws = vae4.alloc_pages_workspace(len(counts))
    vae4.verify_attn_e4m3_resize_pages(t, dev(seq), c, copies, ws, page_tokens=page, status=st)
    want, wc, wcp, wst = plain_resize([list(x) for x in table], list(counts), seq, page)
    assert t.tolist() == want and c.tolist() == wc and copies.tolist() == wcp and int(st) == wst == 0
    # lengths without q: no page is replaced, and nothing is left to do
    vae4.verify_attn_e4m3_resize_pages(t, dev([L for L, _ in seq]), c, copies, ws, page_tokens=page, status=st)
    assert t.tolist() == want and c.tolist() == wc and copies.tolist() == [[-1, -1]] * B and int(st) == 0


@pytest.mark.parametrize("extra", [0, 1, 5, 17])
def test_resize_with_too_few_pages(extra):
    """The first entries in order are served; after others have been freed the same
    call serves the rest."""
    B, cols, page = 9, 12, 16
    table, counts = pool(8, B, cols, extra=extra, share=0.9)
    seq = [(cols * page, cols * page if b % 2 else 5) for b in range(B)]
    t, c, st = dev(table), dev(counts), status()
    copies = torch.empty((B, 2), dtype=torch.int32, device="cuda")
    ws = vae4.alloc_pages_workspace(len(counts))
    short = []
    for _ in range(5):
        vae4.verify_attn_e4m3_resize_pages(t, dev(seq), c, copies, ws, page_tokens=page, status=st.zero_())
        table, counts, wcp, wst = plain_resize(table, counts, seq, page)
        assert t.tolist() == table and c.tolist() == counts and copies.tolist() == wcp and int(st) == wst
        short.append(wst & vae4.STATUS_NO_PAGES)
        seq[seq.index((cols * page, 5))] = (0, 0)
    assert short[0]


@pytest.mark.parametrize("extra", [0, 1, 5000])
def test_resize_of_a_large_pool_that_runs_short(extra):
    """A pool for which the whole GPU is used: too few pages, invalid entries and lengths,
    pages that nothing counts; then a call that finds room."""
    B, cols, page = 130, 300, 16
    table, counts = pool(21, B, cols, extra=extra, share=0.8, kept=7)
    seq = lengths(22, table, page)
    seq[7], seq[8], seq[9] = (cols * page + 1, 1), (5, 6), (-1, 0)
    table[3][1], table[4][0] = len(counts), -2
    t, c, st = dev(table), dev(counts), status()
    copies = torch.empty((B, 2), dtype=torch.int32, device="cuda")
    ws = vae4.alloc_pages_workspace(len(counts))
    for full in (True, False):
        now = [(cols * page, cols * page) if full and b % 3 == 0 else x for b, x in enumerate(seq)]
        vae4.verify_attn_e4m3_resize_pages(t, dev(now), c, copies, ws, page_tokens=page, status=st.zero_())
        table, counts, wcp, wst = plain_resize(table, counts, now, page)
        assert t.tolist() == table and c.tolist() == counts and copies.tolist() == wcp and int(st) == wst
        assert not full or wst & vae4.STATUS_NO_PAGES


def test_counts_below_the_entries():
    """Pages that more entries give up than their counts say: the counts end at zero, which
    is reported, never below it (such a page would be kept for good)."""
    B, cols = 200, 40
    for low in (-2 ** 31, -1, 0, 1, 2):
        counts = [low] * cols + [0] * 5
        table = [list(range(cols)) for _ in range(B)]
        for what in ("release", "replace", "fork"):
            t, c, st = dev(table), dev(counts), status()
            if what == "fork":
                vae4.verify_attn_e4m3_fork_pages(t, c, dev([-1] * B), status=st)
                want, wc, wst = plain_fork([list(x) for x in table], list(counts), [-1] * B)
            else:
                seq = [(0, 0)] * B if what == "release" else [(cols * 16, 16)] * B
                copies, ws = torch.empty((B, 2), dtype=torch.int32, device="cuda"), vae4.alloc_pages_workspace(len(counts))
                vae4.verify_attn_e4m3_resize_pages(t, dev(seq), c, copies, ws, page_tokens=16, status=st)
                want, wc, _, wst = plain_resize([list(x) for x in table], list(counts), seq, 16)
            assert t.tolist() == want and c.tolist() == wc and int(st) == wst, (low, what)


def test_resize_reports():
    table, counts = pool(4, 8, 6, share=0, kept=0)
    table[0][5], table[1][0] = len(counts) + 3, -4
    table[2] = [counts.index(0)] + [-1] * 5
    seq = [(16, 16), (16, 1), (0, 0), (-1, 0), (97, 1), (20, 21), (20, -1), (2 ** 31 - 1, 1)]
    t, c, st = dev(table), dev(counts), status()
    copies = torch.empty((8, 2), dtype=torch.int32, device="cuda")
    vae4.verify_attn_e4m3_resize_pages(t, dev(seq), c, copies, vae4.alloc_pages_workspace(len(counts)),
                                       page_tokens=16, status=st)
    want, wc, wcp, wst = plain_resize([list(x) for x in table], list(counts), seq, 16)
    assert t.tolist() == want and c.tolist() == wc and copies.tolist() == wcp and int(st) == wst
    assert t.tolist()[3:] == table[3:]
    assert wst == (vae4.STATUS_BAD_BLOCK | vae4.STATUS_BAD_COUNT | vae4.STATUS_BAD_LENGTH | vae4.STATUS_BAD_QLEN)


@pytest.mark.parametrize("B,cols", SHAPES)
@pytest.mark.parametrize("m", [1, 13, 5000])
def test_compact(B, cols, m):
    table, counts = pool(3 * B + cols, B, cols, extra=B * cols // 3 + 2)
    t, c, st = dev(table, 3 if m == 13 else 0), dev(counts), status()
    moves = torch.full((m, 2), 55, dtype=torch.int32, device="cuda")
    vae4.verify_attn_e4m3_compact_pages(t, c, moves, status=st)
    want, wc, wm, wst = plain_compact([list(x) for x in table], list(counts), m)
    assert moves.tolist() == wm and t.tolist() == want and c.tolist() == wc and int(st) == wst == 0
    if len([x for x in wm if x[0] >= 0]) < m:  # in order: nothing more to move
        vae4.verify_attn_e4m3_compact_pages(t, c, moves, status=st)
        assert t.tolist() == want and c.tolist() == wc and moves.tolist() == [[-1, -1]] * m


def test_compact_of_odd_pools():
    """No page in use; all in use; kept pages high up, one whose count is the lowest
    number; an invalid entry; no sequence."""
    cases = [([[-1, -1]], [0, 0, 0]), ([[0, 1]], [1, 1]), ([[5, 4]], [0, 0, -1, 0, 1, 1]),
             ([[5, 6]], [0, 0, 0, 0, 0, 1, -2 ** 31]), ([[3, 9, -2]], [0, 0, 0, 1])]
    for table, counts in cases:
        t, c, st = dev(table), dev(counts), status()
        moves = torch.empty((4, 2), dtype=torch.int32, device="cuda")
        vae4.verify_attn_e4m3_compact_pages(t, c, moves, status=st)
        want, wc, wm, wst = plain_compact([list(x) for x in table], list(counts), 4)
        assert (t.tolist(), c.tolist(), moves.tolist(), int(st)) == (want, wc, wm, wst)
    none = torch.empty((0, 3), dtype=torch.int32, device="cuda")
    c, moves = dev([0, 0, 2]), torch.empty((4, 2), dtype=torch.int32, device="cuda")
    vae4.verify_attn_e4m3_compact_pages(none, c, moves)
    assert c.tolist() == [2, 0, 0] and moves.tolist() == [[2, 0]] + [[-1, -1]] * 3


# ---------------------------------------------------------------------------- copying


def caches(n_pages, page, H, D, layout, seed=0):
    g = torch.Generator().manual_seed(seed)
    both = torch.randint(0, 256, (2, n_pages, page, H, D), generator=g, dtype=torch.uint8)
    if layout == "pool":
        kv = both.permute(1, 0, 3, 2, 4).contiguous().cuda()
        return vae4.cache_views(kv)
    if layout == "padded":  # a token stride of 8 bytes' granularity
        out = []
        for w in (0, 1):
            buf = torch.zeros((n_pages, page, H * D + 8), dtype=torch.uint8, device="cuda")
            view = buf[:, :, :H * D].unflatten(2, (H, D))
            view.copy_(both[w])
            out.append(view)
        return tuple(out)
    if layout == "spread":  # heads outermost, space between them and between tokens
        out = []
        for w in (0, 1):
            buf = torch.zeros((H, n_pages, page + 1, D + 16), dtype=torch.uint8, device="cuda")
            view = buf[:, :, :page, :D].permute(1, 2, 0, 3)
            view.copy_(both[w])
            out.append(view)
        return tuple(out)
    return both[0].cuda(), both[1].cuda()


@pytest.mark.parametrize("page,H,D,nb", [(16, 1, 64, 1), (96, 3, 128, 2), (64, 8, 256, 4), (848, 1, 64, 53),
                                        (16, 33, 64, 1)])
@pytest.mark.parametrize("layout", ["pool", "tokens", "padded", "spread"])
@pytest.mark.parametrize("sides", ["none", "scales", "bounds", "both"])
def test_copy(page, H, D, nb, layout, sides):
    n_pages = 23
    k, v = caches(n_pages, page, H, D, layout)
    sc = torch.randn(n_pages, 2, H, nb, device="cuda") if sides in ("scales", "both") else None
    bd = torch.randint(0, 256, (n_pages, H, nb, 2, D), dtype=torch.uint8, device="cuda") if sides in ("bounds", "both") else None
    pairs = [[3, 7], [3, 8], [-1, -1], [22, 0], [5, 5], [11, 22 - 1], [-1, 4], [23, 4], [2, -3], [2, 23]]
    want = [x.clone() if x is not None else None for x in (k, v, sc, bd)]
    for a, b in pairs[:6]:
        for x in want:
            if x is not None and a >= 0:
                x[b] = x[a].clone()
    st = status()
    vae4.verify_attn_e4m3_copy_pages(k, v, dev(pairs), block_scales=sc, k_bounds=bd, status=st)
    for x, y in zip((k, v, sc, bd), want):
        assert x is None or torch.equal(x, y)
    assert int(st) == vae4.STATUS_BAD_BLOCK
    if layout == "padded":
        assert int(k.as_strided((n_pages, page, 8), k.stride()[:2] + (1,), H * D).count_nonzero()) == 0


def test_copy_of_large_pages_and_offsets_past_32_bits():
    """Pages of 65536 tokens, ids whose bytes lie past 2^32 from the base; types of torch."""
    n_pages, page, H, D = 36, 65536, 8, 256
    k = torch.zeros(n_pages, page, H, D, dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    k[35].random_(1, 256), v[35].random_(1, 256)
    e5 = lambda t: t.view(torch.float8_e5m2)  # noqa: E731
    vae4.verify_attn_e4m3_copy_pages(e5(k), e5(v), dev([[35, 34], [0, 1]]))
    for x in (k, v):
        assert torch.equal(x[34], x[35]) and int(x[35].count_nonzero()) == x[35].numel()
        assert not any(bool(x[p].any()) for p in range(34))


# ---------------------------------------------------------------------------- together


def test_a_run_of_steps_beside_caches_of_their_own():
    """Steps of append, fork, resize, copy and compact on one pool: every sequence
    keeps the codes that a cache of its own, without sharing, holds."""
    B, cols, page, blk, H, D = 6, 12, 32, 16, 2, 64
    n_pages = 61
    g = torch.Generator().manual_seed(5)
    r = random.Random(5)
    i32 = lambda *s, v=-1: torch.full(s, v, dtype=torch.int32, device="cuda")  # noqa: E731
    layers = [vae4.cache_views(torch.zeros(n_pages, 2, H, page, D, dtype=torch.uint8, device="cuda")) for _ in range(2)]
    scales = [vae4.alloc_block_scales(n_pages, H, page, blk) for _ in layers]
    bounds = [vae4.alloc_k_bounds(n_pages, H, page, blk, D) for _ in layers]
    table, counts, ws = i32(B, cols), vae4.alloc_ref_counts(n_pages), vae4.alloc_pages_workspace(n_pages)
    copies, moves, st = i32(B, 2), i32(7, 2), status()
    # the same history without sharing: row b of an own cache owns pages b * cols ..
    own = [[x.clone() for x in caches(B * cols, page, H, D, "tokens")] for _ in layers]
    own_sc = [vae4.alloc_block_scales(B * cols, H, page, blk) for _ in layers]
    own_bd = [vae4.alloc_k_bounds(B * cols, H, page, blk, D) for _ in layers]
    own_table = torch.arange(B * cols, dtype=torch.int32, device="cuda").view(B, cols)
    L = [0] * B

    def read(k, v, sc, bd, t, b):
        n, nb = -(-L[b] // page), -(-L[b] // blk)
        pg = t[b, :n].long()
        return [k[pg].flatten(0, 1)[:L[b]], v[pg].flatten(0, 1)[:L[b]],
                sc[pg].permute(1, 2, 0, 3).flatten(2)[:, :, :nb], bd[pg].transpose(0, 1).flatten(1, 2)[:, :nb]]

    for step in range(30):
        parents = list(range(B))
        if step % 3 == 2:
            parents = [r.choice([b, r.randrange(B)]) for b in range(B)]
            vae4.verify_attn_e4m3_fork_pages(table, counts, dev(parents), status=st)
            for l in range(2):
                for x in own[l] + [own_sc[l], own_bd[l]]:
                    y = x.view(B, cols, *x.shape[1:])
                    y.copy_(y[torch.tensor(parents, device="cuda")].clone())
            L = [L[p] for p in parents]
        q = []
        for b in range(B):
            back = r.choice([0, 0, 0, 3])
            if r.random() < 0.1:
                L[b] = 0
            # rejected drafts: a block's scale depends on them, so only whole blocks go
            L[b] = max(0, L[b] - back) // blk * blk if back else L[b]
            n = min(r.choice([0, 1, 5, 8, 40]), cols * page // 3 - L[b])
            q.append(max(n, 0))
            L[b] += q[-1]
        seq = dev(list(zip(L, q)))
        vae4.verify_attn_e4m3_resize_pages(table, seq, counts, copies, ws, page_tokens=page, status=st)
        if step % 4 == 3:
            vae4.verify_attn_e4m3_compact_pages(table, counts, moves, status=st)
        Q = max(max(q), 1)
        for l, (k, v) in enumerate(layers):
            vae4.verify_attn_e4m3_copy_pages(k, v, copies, block_scales=scales[l], k_bounds=bounds[l], status=st)
            if step % 4 == 3:
                vae4.verify_attn_e4m3_copy_pages(k, v, moves, block_scales=scales[l], k_bounds=bounds[l], status=st)
            kn, vn = [torch.randn(B, Q, H, D, generator=g).half().cuda() for _ in range(2)]
            vae4.verify_attn_e4m3_append(kn, vn, k, v, table, seq, scales[l], k_bounds=bounds[l], status=st)
            vae4.verify_attn_e4m3_append(kn, vn, *own[l], own_table, seq, own_sc[l], k_bounds=own_bd[l], status=st)
            for b in range(B):
                got = read(k, v, scales[l], bounds[l], table, b)
                for x, y in zip(got, read(*own[l], own_sc[l], own_bd[l], own_table, b)):
                    assert torch.equal(x, y), (step, l, b)
        assert int(st) == 0
        # the counts are those of the table, and what is freed is free
        ids = [e for row in table.tolist() for e in row if e >= 0]
        assert counts.tolist() == [ids.count(x) for x in range(n_pages)]
        assert [sum(e >= 0 for e in row) for row in table.tolist()] == [-(-x // page) for x in L]


def test_calls_in_a_captured_graph():
    """Fork, resize, copy and compact captured once and replayed on other contents."""
    B, cols, page, H, D = 5, 20, 16, 1, 64
    pools = [pool(s, B, cols, extra=B * cols, share=0.8) for s in range(3)]
    n_pages = max(len(c) for _, c in pools)
    table, counts = torch.full((B, cols), -1, dtype=torch.int32, device="cuda"), vae4.alloc_ref_counts(n_pages)
    parents = torch.arange(B, dtype=torch.int32, device="cuda")
    seq, copies = [torch.zeros(B, 2, dtype=torch.int32, device="cuda") for _ in range(2)]
    moves = torch.zeros(50, 2, dtype=torch.int32, device="cuda")
    ws, st = vae4.alloc_pages_workspace(n_pages), status()
    k, v = caches(n_pages, page, H, D, "tokens")

    def step():
        vae4.verify_attn_e4m3_fork_pages(table, counts, parents, status=st)
        vae4.verify_attn_e4m3_resize_pages(table, seq, counts, copies, ws, page_tokens=page, status=st)
        vae4.verify_attn_e4m3_copy_pages(k, v, copies, status=st)
        vae4.verify_attn_e4m3_compact_pages(table, counts, moves, status=st)
        vae4.verify_attn_e4m3_copy_pages(k, v, moves, status=st)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for s, (t, c) in enumerate(pools):
        c = c + [0] * (n_pages - len(c))
        par = [(b + s) % B if b else 0 for b in range(B)]
        t2, c2, f = plain_fork([list(x) for x in t], list(c), par)
        sq = lengths(s, t2, page)
        table.copy_(dev(t)), counts.copy_(dev(c)), parents.copy_(dev(par)), seq.copy_(dev(sq))
        wk = k.clone()
        graph.replay()
        t2, c2, wcp, f2 = plain_resize(t2, c2, sq, page)
        t2, c2, wm, f3 = plain_compact(t2, c2, 50)
        assert table.tolist() == t2 and counts.tolist() == c2 and copies.tolist() == wcp and moves.tolist() == wm
        assert int(st) == (f | f2 | f3) == 0
        for a, b in wcp + wm:
            if a >= 0:
                wk[b] = wk[a].clone()
        assert torch.equal(k, wk)


def test_another_stream():
    table, counts = pool(1, 31, 40, extra=31 * 40)
    seq = lengths(1, table, 16)
    s = torch.cuda.Stream()
    t, c, q = dev(table), dev(counts), dev(seq)
    copies, ws = torch.empty((31, 2), dtype=torch.int32, device="cuda"), vae4.alloc_pages_workspace(len(counts))
    s.wait_stream(torch.cuda.current_stream())
    vae4.verify_attn_e4m3_resize_pages(t, q, c, copies, ws, page_tokens=16, stream=s)
    s.synchronize()
    want, wc, wcp, _ = plain_resize(table, counts, seq, 16)
    assert t.tolist() == want and c.tolist() == wc and copies.tolist() == wcp
