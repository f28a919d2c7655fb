"""Cases of two kinds of operators around the paged FP8 cache: attention of chunks of new tokens, and the pages' lives.

chunk: attention of a chunk of q new tokens of each sequence, any number of them, over the paged cache
that already holds them: query i of a sequence (L, q) sees the keys 0 .. L - q + i.  The cache is K and V
[n_pages][page][Hkv][D] in FP8 with FP32 scales: one for every `block` tokens and KV head ([n_pages][2]
[Hkv][page / block], index 0: K, 1: V) or one per KV head ([Hkv][2]).

pages: a pool is a block table [B][columns] of page ids (-1: none) and a count for every page of the
entries that hold it (0: free; below 0: kept, neither handed out nor freed).  copy moves pages of a
cache; fork makes rows of the table equal to other rows; resize gives every sequence the pages of its
length, those of its new tokens its own; compact moves the pages in use to the low ids.

`own = False` computes every operator with elementary torch operations, `own = True` through the package.
"""
import math

import torch

own = False

NEG = float("-inf")
FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
KIND = {"f16": torch.float16, "bf16": torch.bfloat16}
FAR = 1 << 30


def listed():
    return [
        # the last tokens of a short prompt: the smallest call, a launch's latency
        case("chunk_short", "chunk", B=1, q=32, Hq=2, Hkv=1, D=64, L=1024, page=16, block=16, scaled="head"),
        # a whole prompt at once
        case("chunk_prompt", "chunk", B=1, q=8192, Hq=64, Hkv=8, D=128, L=8192, page=64, block=64, dtype="bf16"),
        # a chunk at the end of a long context
        case("chunk_long", "chunk", B=1, q=2048, Hq=6, Hkv=1, D=256, L=262144, page=16, block=16),
        # a step of a server: chunks of prompts beside single tokens, an odd page size
        case("chunk_mixed", "chunk", B=24, q=509, Hq=24, Hkv=8, D=128, L=32749, page=96, block=48, ragged=1, layout="tokens"),
        # the partly filled page of one forked sequence: the smallest copy
        case("copy_one", "copy", n=1, n_pages=64, Hkv=1, D=64, page=16, block=16),
        # a compaction's moves, with the bounds that sparse attention reads
        case("copy_many", "copy", n=901, n_pages=2048, Hkv=8, D=128, page=64, block=64, bounds=1, layout="tokens"),
        # a prompt's row taken over by the samples that continue it
        case("fork_samples", "fork", B=8, L=1024, page=16),
        # a step of beam search: rows that change places, and some that end
        case("fork_beams", "fork", B=256, L=32749, page=16, share=4),
        # room for a step's tokens, a small batch
        case("resize_step", "resize", B=8, L=1024, page=16, q=8),
        # a server's step: sequences that grow, end, begin, or give rejected drafts back
        case("resize_batch", "resize", B=256, L=32749, page=16, q=8, share=4),
        # a small pool in order
        case("compact_small", "compact", B=8, L=1024, page=16, n=64),
        # the pool of long contexts in order, a bounded number of moves
        case("compact_large", "compact", B=32, L=262144, page=16, share=2, n=16384),
    ]


def case(name, op, **kw):
    c = dict(name=name, op=op, B=1, q=1, Hq=0, Hkv=1, D=0, L=0, page=16, block=16, n=0, n_pages=0, share=1, ragged=0,
             bounds=0, scaled="block", fmt="e4m3", dtype="f16", layout="pool")
    c.update(kw)
    return c


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        for key in w:
            most[c["op"], key] = max(most.get((c["op"], key), 0), w[key])
    spread = lambda a, b: int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))  # noqa: E731
    op = rng.choice(["chunk", "chunk", "chunk", "copy", "fork", "resize", "compact"])
    while True:
        block = 16 * rng.choice([1, 1, 2, 3, 4, 4, 8])
        page = block * rng.choice([1, 1, 2, 4])
        if op in ("chunk", "copy"):
            kv = rng.choice([1, 1, 2, 3, 4, 8])
            c = case(None, op, Hkv=kv, D=rng.choice([64, 128, 256]), page=page, block=block,
                     fmt=rng.choice(["e4m3", "e4m3", "e4m3", "e5m2"]), layout=rng.choice(["pool", "tokens"]))
        else:
            c = case(None, op, B=spread(1, 256), L=spread(16, 262144), page=page, share=rng.choice([1, 2, 4, 7]))
        if op == "chunk":
            c.update(B=spread(1, 24), q=spread(1, 8192), Hq=kv * rng.choice([1, 2, 3, 4, 5, 6, 8, 12, 16]),
                     dtype=rng.choice(["f16", "bf16"]), ragged=rng.randrange(2), scaled=rng.choice(["block", "block", "head"]))
            c["L"] = max(spread(16, 262144), c["q"])
            if c["B"] * c["L"] * kv * c["D"] > 600e6 or c["L"] * c["q"] * c["Hq"] > 4e9 * c["B"]:
                continue
        elif op == "copy":
            c.update(n=spread(1, 1024), bounds=rng.randrange(2))
            c["n_pages"] = 2 * c["n"] + spread(8, 256)
            if c["n_pages"] * page * kv * c["D"] > 150e6:
                continue
        elif op == "resize":
            c["q"] = rng.choice([1, 1, 2, 5, 8, 16])
        elif op == "compact":
            c["n"] = spread(1, 16384)
        w = work(c)
        if all(w[key] <= most[op, key] for key in w):
            c.pop("name")
            return c


def lengths(c):
    """Of a chunk case: (L, q) of every sequence, from the case alone."""
    out = []
    for b in range(c["B"]):
        q, part = c["q"], 1.0
        if c["ragged"]:
            q = (q, 1, max(1, q // 2))[b % 3]
            part = 1.0 if b == 0 else 0.3 + 0.7 * ((0.6180339887 * b) % 1.0)
        out.append((max(int(c["L"] * part), q), q))
    return out


def held(c):
    """Of a pool: tokens of every sequence before the call, those whose pages it shares with the first of its group."""
    out = []
    for b in range(c["B"]):
        part = 1.0 if b == 0 else 0.3 + 0.7 * ((0.6180339887 * b) % 1.0)
        L = max(int(c["L"] * part), 1)
        if c["op"] == "fork" and c["share"] == 1 and b > c["B"] // 2:
            L = 0  # rows that a sequence is going to be forked into
        if c["op"] == "resize" and b % 5 == 3:
            L = 0  # sequences that are about to begin
        lead = out[b - b % c["share"]][0] if b % c["share"] else 0
        out.append((L, min(L, lead) // 2 if b % c["share"] and b % 2 else min(L, lead)))
    return out


def wanted(c):
    """Of a resize case: (L, q) of every sequence for the step to come."""
    out = []
    for b, (L, _) in enumerate(held(c)):
        kind = b % 5
        if kind == 2 and b % 10 == 2:
            out.append((0, 0))  # ended
        elif kind == 3:
            n = min(c["L"], 17 + 37 * b % 4001)
            out.append((n, n))  # a new prompt
        else:
            back = c["q"] // 2 if kind == 1 else 0  # drafts that were rejected
            n = min(max(L - back, 0) + c["q"], columns(c) * c["page"])
            out.append((n, min(c["q"], n)))
    return out


def cells(n, size):
    return -(-n // size)


def columns(c):
    return cells(c["L"] + (c["q"] if c["op"] == "resize" else 0), c["page"])


def used_pages(c):
    return sum(cells(L, c["page"]) - min(cells(s, c["page"]), cells(L, c["page"])) for L, s in held(c))


def pool_pages(c):
    """Pages of the pool: those in use, and those that a step can take."""
    new = sum(cells(L, c["page"]) for L, q in wanted(c) if L == q) if c["op"] == "resize" else 0
    return cells(used_pages(c) * 5 // 4 + new + 2 * c["B"] + 16, 16) * 16


def work(c):
    """Bytes that have to move and operations that have to be done, each input once and each output once."""
    op, D, H = c["op"], c["D"], c["Hkv"]
    nbytes = flops = 0
    if op == "chunk":
        for L, n in lengths(c):
            nbytes += 2 * H * L * D + 2 * n * c["Hq"] * D * 2 + 4 * cells(L, c["page"])
            nbytes += cells(L, c["block"]) * H * 8 if c["scaled"] == "block" else 0
            flops += 4 * c["Hq"] * D * (n * (L - n) + n * (n + 1) // 2)
    elif op == "copy":
        one = 2 * H * c["page"] * D + (c["page"] // c["block"]) * H * (8 + (2 * D if c["bounds"] else 0))
        nbytes, flops = c["n"] * (2 * one + 8), c["n"] * H * c["page"] * D
    else:
        table, counts = 4 * c["B"] * columns(c), 4 * pool_pages(c)
        nbytes = table + counts + (table + 4 * c["B"] if op == "fork" else 8 * c["n"] if op == "compact" else 16 * c["B"])
        flops = nbytes // 4
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------------------- inputs


def cache(c, n_pages, gen):
    """K and V caches of random values with outliers and blocks of different size, and their scales."""
    page, H, D, blk = c["page"], c["Hkv"], c["D"], c["block"]
    kind, top = FP8[c["fmt"]]
    nb, pool = page // blk, c["layout"] == "pool"
    both = torch.empty((n_pages, 2, H, page, D) if pool else (2, n_pages, page, H, D), dtype=torch.uint8, device="cuda")
    views = [both[:, s].transpose(1, 2) if pool else both[s] for s in (0, 1)]
    scales = torch.empty(n_pages, 2, H, nb, device="cuda")
    head = 0.02 * torch.exp(0.5 * torch.randn(H, 2, generator=gen, device="cuda"))
    step = max(1, (1 << 26) // (page * H * D))
    for s in (0, 1):
        for p0 in range(0, n_pages, step):
            n = min(step, n_pages - p0)
            x = torch.randn(n, nb, blk, H, D, generator=gen, device="cuda")
            x *= torch.exp(0.5 * torch.randn(n, nb, 1, H, 1, generator=gen, device="cuda"))
            x *= 1 + 7 * (torch.rand(n, nb, 1, H, D, generator=gen, device="cuda") < 0.01)  # channels that stand out
            sc = x.abs().amax((2, 4)) / top
            if c["op"] == "chunk" and c["scaled"] == "head":
                sc = head[:, s].expand(n, nb, H)
            x = (x / sc[:, :, None, :, None]).clamp(-top, top).to(kind).view(torch.uint8)
            views[s][p0:p0 + n] = x.reshape(n, page, H, D)
            scales[p0:p0 + n, s] = sc.transpose(1, 2)
    return views[0], views[1], scales, head


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return globals()["prepare_" + (c["op"] if c["op"] in ("chunk", "copy") else "pool")](c, gen)


def prepare_chunk(c, gen):
    pairs = lengths(c)
    top = max(L for L, _ in pairs)
    st = {"case": dict(c), "pairs": pairs, "top": top, "seq": torch.tensor(pairs, dtype=torch.int32, device="cuda")}
    per = [cells(L, c["page"]) for L, _ in pairs]
    n_pages = sum(per) + 3
    order = torch.randperm(n_pages, generator=gen, device="cuda").int()
    st["table"] = torch.full((c["B"], max(per)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(per):
        st["table"][b, :n] = order[at:at + n]
        at += n
    st["k_cache"], st["v_cache"], scales, head = cache(c, n_pages, gen)
    st["scales"] = scales if c["scaled"] == "block" else head
    q = torch.randn(c["B"], c["q"], c["Hq"], c["D"], generator=gen, device="cuda")
    q *= torch.exp(0.5 * torch.randn(c["B"], 1, c["Hq"], 1, generator=gen, device="cuda"))  # heads of different sharpness
    st["q"] = q.to(KIND[c["dtype"]])
    st["out"] = torch.zeros_like(st["q"])
    return st


def prepare_copy(c, gen):
    st = {"case": dict(c)}
    st["k_cache"], st["v_cache"], st["scales"], _ = cache(c, c["n_pages"], gen)
    order = torch.randperm(c["n_pages"], generator=gen, device="cuda").int()
    st["pairs"] = order[:2 * c["n"]].view(2, c["n"]).T.contiguous()
    st["bounds"] = None
    if c["bounds"]:
        nb, (kind, top) = c["page"] // c["block"], FP8[c["fmt"]]
        x = torch.randn(c["n_pages"], c["Hkv"], nb, 2, c["D"], generator=gen, device="cuda") * 100
        st["bounds"] = x.clamp(-top, top).to(kind).view(torch.uint8)
    return st


def prepare_pool(c, gen):
    B, cols, n_pages = c["B"], columns(c), pool_pages(c)
    had = held(c)
    P = torch.tensor([cells(L, c["page"]) for L, _ in had], device="cuda")[:, None]
    S = torch.tensor([cells(s, c["page"]) for _, s in had], device="cuda")[:, None]
    j = torch.arange(cols, device="cuda")
    mine = (j < P) & (j >= S)
    order = torch.randperm(n_pages, generator=gen, device="cuda")
    rank = mine.flatten().long().cumsum(0).view(B, cols) - 1
    table = torch.where(mine, order[rank.clamp_min(0)], -1)
    lead = torch.arange(B, device="cuda") // c["share"] * c["share"]
    table = torch.where((j < P) & ~mine, table[lead], table)
    counts = torch.zeros(n_pages, dtype=torch.int64, device="cuda")
    counts.index_add_(0, table.clamp_min(0).flatten(), (table >= 0).long().flatten())
    counts[order[used_pages(c):used_pages(c) + 2]] = -1  # pages that are kept
    st = {"case": dict(c), "was": torch.cat([counts, table.flatten()]).int()}
    # one buffer, so that a pass can begin with the pool as it was
    st["pool"] = st["was"].clone()
    st["counts"], st["table"] = st["pool"][:n_pages], st["pool"][n_pages:].view(B, cols)
    if c["op"] == "fork":
        if c["share"] == 1:  # the rows of the second half follow one of the first
            parents = torch.arange(B, device="cuda")
            some = torch.randint(0, B // 2 + 1, (B,), generator=gen, device="cuda")
            parents = torch.where(parents > B // 2, some, parents)
        else:
            parents = lead + torch.randint(0, c["share"], (B,), generator=gen, device="cuda")
            parents = parents.clamp_max(B - 1)
            ends = torch.rand(B, generator=gen, device="cuda") < 0.05
            parents = torch.where(ends, -1, parents)
        st["parents"] = parents.int()
    elif c["op"] == "resize":
        st["seq"] = torch.tensor(wanted(c), dtype=torch.int32, device="cuda")
        st["copies"] = torch.full((B, 2), -7, dtype=torch.int32, device="cuda")
    else:
        st["moves"] = torch.full((c["n"], 2), -7, dtype=torch.int32, device="cuda")
    return st


# ---------------------------------------------------------------------------- a pass


def run(st):
    if "pool" in st:
        st["pool"].copy_(st["was"])
    return globals()[("own_" if own else "plain_") + st["case"]["op"]](st)


def fp8(t, c):
    return t.view(FP8[c["fmt"]][0])


def plain_values(st, c, b, L, kind):
    """K and V [Hkv][L][D] of sequence b."""
    page, blk = c["page"], c["block"]
    t = torch.arange(L, device="cuda")
    pg, slot = st["table"][b].long()[t // page], t % page
    out = []
    for s, x in ((0, st["k_cache"]), (1, st["v_cache"])):
        y = fp8(x[pg, slot], c).to(kind)  # [L][H][D]
        if c["scaled"] == "block":
            y = y * st["scales"][pg, s, :, slot // blk].to(kind)[:, :, None]
        else:
            y = y * st["scales"][:, s].to(kind)[:, None]
        out.append(y.transpose(0, 1))
    return out


def plain_chunk(st):
    c = st["case"]
    H, G, D = c["Hkv"], c["Hq"] // c["Hkv"], c["D"]
    for b, (L, n) in enumerate(st["pairs"]):
        K, V = plain_values(st, c, b, L, torch.float32)
        step = max(1, (1 << 28) // (c["Hq"] * L))
        for i0 in range(0, n, step):
            m = min(step, n - i0)
            top = L - n + i0 + m  # keys that the last of these queries sees
            x = st["q"][b, i0:i0 + m].float().view(m, H, G, D).permute(1, 0, 2, 3).reshape(H, m * G, D)
            z = torch.matmul(x, K[:, :top].transpose(1, 2)).view(H, m, G, top) / math.sqrt(D)
            see = L - n + i0 + torch.arange(m, device="cuda")
            z = z.masked_fill(torch.arange(top, device="cuda") > see[:, None, None], NEG)
            z = torch.exp(z - z.amax(-1, keepdim=True))
            o = torch.matmul(z.view(H, m * G, top), V[:, :top]).view(H, m, G, D) / z.sum(-1, keepdim=True)
            st["out"][b, i0:i0 + m] = o.permute(1, 0, 2, 3).reshape(m, H * G, D).to(st["out"].dtype)
    return st["out"]


def plain_copy(st):
    src, dst = st["pairs"][:, 0].long(), st["pairs"][:, 1].long()
    for x in (st["k_cache"], st["v_cache"], st["scales"], st["bounds"]):
        if x is not None:
            x[dst] = x[src]
    return outputs_copy(st)


def outputs_copy(st):
    c = st["case"]
    out = {"k_cache": fp8(st["k_cache"], c), "v_cache": fp8(st["v_cache"], c), "scales": st["scales"]}
    if st["bounds"] is not None:
        out["bounds"] = fp8(st["bounds"], c)
    return out


def add_counts(counts, pages, what):
    """counts[pages] += what, but for pages that are kept."""
    at = pages.clamp_min(0).flatten()
    what = torch.where((pages.flatten() >= 0) & (counts[at] > 0), what.flatten().int(), 0)
    counts.index_add_(0, at, what)


def plain_fork(st):
    T, par = st["table"], st["parents"].long()
    rows = torch.arange(T.shape[0], device="cuda")
    kids = (par == rows[:, None]).sum(1)
    add_counts(st["counts"], T.long(), (kids - 1)[:, None].expand(T.shape))
    T.copy_(torch.where(par[:, None] >= 0, T[par.clamp_min(0)], -1))
    return {"table": T, "counts": st["counts"]}


def plain_resize(st):
    page, T, counts = st["case"]["page"], st["table"], st["counts"]
    L, q = st["seq"][:, 0, None].long(), st["seq"][:, 1, None].long()
    j = torch.arange(T.shape[1], device="cuda")
    n, first = (L + page - 1) // page, (L - q) // page
    old = T.long()
    gone = (old >= 0) & (j >= n)
    add_counts(counts, torch.where(gone, old, -1), torch.full_like(old, -1))
    old = torch.where(gone, -1, old)
    have = counts[old.clamp_min(0)]
    shared = (old >= 0) & ((have > 1) | (have < 0)) & (j >= first) & (q > 0)
    need = (j < n) & ((old < 0) | shared)
    ids = torch.arange(counts.shape[0], device="cuda")
    free = torch.where(counts == 0, ids, FAR).sort().values
    rank = (need.flatten().long().cumsum(0) - 1).view(T.shape).clamp(0, counts.shape[0] - 1)
    new = free[rank]
    served = need & (new < FAR) & (need.flatten().long().cumsum(0) <= counts.shape[0]).view(T.shape)
    taken = torch.where(served, new, 0).flatten()
    add_counts(counts, torch.where(served, old, -1), torch.full_like(old, -1))
    counts.index_add_(0, taken, served.flatten().int())
    keeps = served & (old >= 0) & (j == first) & ((L - q) % page != 0)
    st["copies"][:, 0] = torch.where(keeps, old, -1).amax(1)
    st["copies"][:, 1] = torch.where(keeps, new, -1).amax(1)
    T.copy_(torch.where(served, new, old))
    return {"table": T, "counts": counts, "copies": st["copies"]}


def plain_compact(st):
    T, counts, M = st["table"], st["counts"], st["moves"].shape[0]
    n_pages = counts.shape[0]
    ids = torch.arange(n_pages, device="cuda")
    n = (counts != 0).sum()
    dst = torch.where((counts == 0) & (ids < n), ids, FAR).sort().values[:M]
    src = torch.where((counts > 0) & (ids >= n), ids, -1).sort(descending=True).values[:M]
    ok = (dst < FAR) & (src >= 0)
    src, dst = torch.where(ok, src, -1), torch.where(ok, dst, -1)
    st["moves"].fill_(-1)
    st["moves"][:src.shape[0], 0] = src
    st["moves"][:src.shape[0], 1] = dst
    goes = torch.arange(n_pages + 1, device="cuda")
    goes[torch.where(ok, src, n_pages)] = torch.where(ok, dst, n_pages)
    T.copy_(torch.where(T >= 0, goes[T.clamp_min(0).long()], T))
    more = torch.cat([counts, counts.new_zeros(1)])
    was = torch.where(ok, more[src], 0)
    more[torch.where(ok, dst, n_pages)] = was
    more[torch.where(ok, src, n_pages)] = 0
    counts.copy_(more[:n_pages])
    return {"table": T, "counts": counts, "moves": st["moves"]}


# ---------------------------------------------------------------------------- the package's calls


def own_chunk(st):
    import fp8_paged_attention_e4m3_gb300 as vae4
    c = st["case"]
    if "ws" not in st:  # a program keeps its workspace from step to step
        st["ws"] = vae4.alloc_chunk_workspace(c["B"], c["Hq"], c["Hkv"], c["q"], c["D"], st["top"])
    return vae4.verify_attn_e4m3_chunk(st["q"], st["k_cache"], st["v_cache"], st["table"], st["seq"], st["scales"],
                                       st["out"], st["ws"], max_seq_len=st["top"],
                                       flags=vae4.FLAG_KV_E5M2 if c["fmt"] == "e5m2" else 0)


def own_copy(st):
    import fp8_paged_attention_e4m3_gb300 as vae4
    vae4.verify_attn_e4m3_copy_pages(st["k_cache"], st["v_cache"], st["pairs"], block_scales=st["scales"],
                                     k_bounds=st["bounds"])
    return outputs_copy(st)


def own_fork(st):
    import fp8_paged_attention_e4m3_gb300 as vae4
    vae4.verify_attn_e4m3_fork_pages(st["table"], st["counts"], st["parents"])
    return {"table": st["table"], "counts": st["counts"]}


def own_resize(st):
    import fp8_paged_attention_e4m3_gb300 as vae4
    if "ws" not in st:
        st["ws"] = vae4.alloc_pages_workspace(st["counts"].shape[0])
    vae4.verify_attn_e4m3_resize_pages(st["table"], st["seq"], st["counts"], st["copies"], st["ws"],
                                       page_tokens=st["case"]["page"])
    return {"table": st["table"], "counts": st["counts"], "copies": st["copies"]}


def own_compact(st):
    import fp8_paged_attention_e4m3_gb300 as vae4
    vae4.verify_attn_e4m3_compact_pages(st["table"], st["counts"], st["moves"])
    return {"table": st["table"], "counts": st["counts"], "moves": st["moves"]}


# ---------------------------------------------------------------------------- 64 bits, from the definitions


def exact(c, seed):
    if c["op"] == "chunk":
        return exact_chunk(c, prepare(c, seed))
    if c["op"] == "copy":
        return exact_copy(c, prepare(c, seed))
    return None  # whole numbers


def exact_chunk(c, st):
    G, D, page, blk = c["Hq"] // c["Hkv"], c["D"], c["page"], c["block"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for b, (L, n) in enumerate(lengths(c)):
        pages = st["table"][b, :cells(L, page)].long()
        for h in range(c["Hkv"]):
            kv = []
            for s, x in ((0, st["k_cache"]), (1, st["v_cache"])):
                y = x[pages, :, h].contiguous().view(FP8[c["fmt"]][0]).double()  # [pages][page][D]
                if c["scaled"] == "block":
                    y = y * st["scales"][pages, s, h].double().repeat_interleave(blk, 1)[..., None]
                else:
                    y = y * st["scales"][h, s].double()
                kv.append(y.flatten(0, 1)[:L])
            step = max(1, (1 << 28) // (G * L))
            for i0 in range(0, n, step):
                x = st["q"][b, i0:min(i0 + step, n), h * G:(h + 1) * G].double()
                z = torch.einsum("igd,td->gti", x, kv[0]) / math.sqrt(D)
                i = L - n + i0 + torch.arange(x.shape[0], device="cuda")
                z[:, torch.arange(L, device="cuda")[:, None] > i] = NEG
                w = torch.softmax(z, 1)
                out[b, i0:i0 + x.shape[0], h * G:(h + 1) * G] = torch.einsum("gti,td->igd", w, kv[1])
    return out


def exact_copy(c, st):
    out = {}
    for name, x in (("k_cache", st["k_cache"]), ("v_cache", st["v_cache"]), ("scales", st["scales"]), ("bounds", st["bounds"])):
        if x is not None:
            x = x if name == "scales" else fp8(x, c)
            from_page = torch.arange(c["n_pages"], device="cuda")
            from_page[st["pairs"][:, 1].long()] = st["pairs"][:, 0].long()
            out[name] = torch.stack([x[p].double() for p in from_page.tolist()])
    return out
