"""Cases of the block-scaled cache's operators: append, attention, block scores, block choice, sparse attention.

The cache is paged FP8 (E4M3 or E5M2), K and V [n_pages][page][Hkv][D], with one FP32 scale for every
`block` tokens and KV head, [n_pages][2][Hkv][page / block] (index 0: K, 1: V).  `k_bounds` [n_pages][Hkv]
[page / block][2][D] holds, in the codes of the cache, the smallest and the largest K of a block for
each channel.  Lengths are (L, q) pairs: L tokens of which the last q are the step's own.

`own = False` computes every operator with elementary torch operations, `own = True` through the package.
"""
import math

import torch

own = False

NEG = float("-inf")
FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0, 8), "e5m2": (torch.float8_e5m2, 57344.0, 15)}


def listed():
    return [
        # one new token for each of two sequences: the smallest write, a launch's latency
        case("append_token", "append", B=2, q=1, Hkv=1, D=64, past=100, page=16, block=16),
        # the draft tokens of a verify step, ragged batch, with the bounds that sparse attention reads
        case("append_drafts", "append", B=16, q=8, Hkv=2, D=256, past=5000, page=16, block=16, ragged=1, bounds=1, layout="tokens"),
        # two prompts written at once, starting inside a block
        case("append_prompt", "append", B=2, q=16384, Hkv=8, D=128, past=37, page=64, block=64, bounds=1, dtype="bf16"),
        # verification of eight drafts over a short context
        case("attend_short", "attend", B=1, q=8, Hq=2, Hkv=1, D=64, L=1024, page=16, block=16),
        # verification of eight drafts over a long context, one sequence
        case("attend_long", "attend", B=1, q=8, Hq=6, Hkv=1, D=256, L=262144, page=16, block=16),
        # single-token decoding of a ragged batch, an odd page size
        case("attend_batch", "attend", B=32, q=1, Hq=64, Hkv=8, D=128, L=32749, page=96, block=48, ragged=1, layout="tokens"),
        # the scores of every block of a long context for eight drafts
        case("scores_long", "scores", B=1, q=8, Hq=12, Hkv=2, D=256, L=262144, page=64, block=64),
        # the same for single tokens of a batch
        case("scores_batch", "scores", B=16, q=1, Hq=64, Hkv=8, D=128, L=131072, page=64, block=32, ragged=1),
        # the choice of blocks for eight drafts of a long context
        case("select_long", "select", B=1, q=8, Hkv=2, L=262144, block=64, k=64, sink=1, local=2),
        # the same for single tokens of a batch, from many small blocks
        case("select_batch", "select", B=32, q=1, Hkv=8, L=262139, block=16, k=255, sink=4, local=4, ragged=1),
        # verification of eight drafts over chosen blocks of a long context; the drafts share most blocks
        case("sparse_verify", "sparse", B=1, q=8, Hq=6, Hkv=1, D=256, L=262144, page=16, block=16, k=128, apart=16),
        # single-token decoding of a batch over chosen blocks
        case("sparse_batch", "sparse", B=16, q=1, Hq=64, Hkv=8, D=128, L=65531, page=64, block=64, k=64, ragged=1, layout="tokens"),
    ]


def case(name, op, **kw):
    c = dict(name=name, op=op, B=1, q=1, Hq=0, Hkv=1, D=0, L=0, past=0, page=0, block=16, k=0, sink=0, local=1,
             apart=0, ragged=0, bounds=0, fmt="e4m3", dtype="f16", layout="pool")
    c.update(kw)
    return c


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        for key in w:
            most[c["op"], key] = max(most.get((c["op"], key), 0), w[key])
    while True:
        op = rng.choice(["append", "attend", "scores", "select", "sparse"])
        spread = lambda a, b: int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))  # noqa: E731
        block = 16 * rng.choice([1, 1, 2, 3, 4, 4, 8])
        D = rng.choice([64, 128, 256])
        kv = rng.choice([1, 1, 2, 3, 4, 8])
        q = rng.choice([1, 1, 2, 3, 5, 8, 8, 16])
        group = rng.choice([g for g in (1, 2, 3, 4, 5, 6, 8, 12, 16) if g * q <= 96])
        c = case(None, op, B=spread(1, 32), q=q, Hq=group * kv, Hkv=kv, D=D, L=spread(16, 262144),
                 page=block * rng.choice([1, 1, 2, 4]), block=block, ragged=rng.randrange(2),
                 fmt=rng.choice(["e4m3", "e4m3", "e4m3", "e5m2"]), layout=rng.choice(["pool", "tokens"]))
        if op == "append":
            c.update(Hq=0, L=0, past=spread(1, 6000) - 1, q=spread(1, 16384), bounds=rng.randrange(2), dtype=rng.choice(["f16", "bf16"]))
        else:
            c["L"] = max(c["L"], 4 * q)
        if op in ("select", "sparse"):
            n = shortest(c) // block
            if n < 4:
                continue
            c["sink"], c["local"] = (rng.randrange(4), rng.randrange(1, 5)) if op == "select" else (0, 1)
            c["k"] = max(c["sink"] + c["local"], min(spread(4, 512), max(4, n)))
            if op == "select":
                c.update(Hq=0, D=0, page=0, fmt="e4m3", layout="pool")
            else:
                c["apart"] = rng.randrange(1 + max(0, min(c["k"] - 1, (n - c["k"]) // q)))
                if c["k"] + (q - 1) * c["apart"] > n:
                    continue
        w = work(c)
        if all(w[key] <= most[op, key] for key in w) and w["bytes"] > 0:
            c.pop("name")
            return c


def lengths(c):
    """(L, q) of every sequence, from the case alone."""
    top = c["past"] + c["q"] if c["op"] == "append" else c["L"]
    out = []
    for b in range(c["B"]):
        q = c["q"]
        if c["ragged"] and b % 3 == 1:
            q = max(1, q // 2)
        part = 1.0 if b == 0 or not c["ragged"] else 0.3 + 0.7 * ((0.6180339887 * b) % 1.0)
        out.append((max(int(top * part), q), q))
    return out


def shortest(c):
    return min(L for L, _ in lengths(c))


def blocks(n, block):
    return -(-n // block)


def work(c):
    """Bytes that have to move and operations that have to be done, each input once and each output once."""
    D, H, q, blk, op = c["D"], c["Hkv"], c["q"], c["block"], c["op"]
    nbytes = flops = 0
    for L, n in lengths(c):
        if op == "append":
            old = (L - n) % blk  # tokens of the first block that stay
            touched = blocks(L, blk) - (L - n) // blk
            nbytes += 2 * H * n * D * 3 + touched * H * 8 + (H * old * D if c["bounds"] else 0)
            nbytes += touched * H * 2 * D if c["bounds"] else 0
            flops += 2 * H * n * D * 3
        elif op == "attend":
            nbytes += 2 * H * L * D + blocks(L, blk) * H * 8 + 2 * n * c["Hq"] * D * 2
            flops += 4 * c["Hq"] * n * L * D
        elif op == "scores":
            nbytes += blocks(L, blk) * H * (2 * D + 4 + 4 * n) + n * c["Hq"] * D * 2
            flops += 4 * c["Hq"] * n * blocks(L, blk) * D
        elif op == "select":
            nbytes += H * n * (4 * blocks(L, blk) + 4 * c["k"])
            flops += H * n * blocks(L, blk) * 4
        else:
            nbytes += H * (c["k"] + (n - 1) * c["apart"]) * (blk * 2 * D + 8) + 4 * H * n * c["k"] + 2 * n * c["Hq"] * D * 2
            flops += 4 * c["Hq"] * n * c["k"] * blk * D
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------------------- inputs


def pow2_scale(amax, fmt):
    """The smallest power of two s with amax <= s * (largest value of the format), within 2^-30 .. 2^30."""
    _, top, _ = FP8[fmt]
    m, e = torch.frexp(amax.double())  # amax = m * 2^e, m in [0.5, 1); top = 0.875 * 2^et
    et = math.frexp(top)[1]
    e = torch.where(amax > 0, e - et + (m > 0.875).int(), torch.full_like(e, -30)).clamp(-30, 30)
    return torch.ldexp(torch.ones_like(m), e).float()


def cache(c, n_pages, gen, pow2):
    """K and V caches of random values with outliers and blocks of different size, and their scales."""
    page, H, D, blk = c["page"], c["Hkv"], c["D"], c["block"]
    kind, top, _ = FP8[c["fmt"]]
    nb = page // blk
    pool = c["layout"] == "pool"
    shape = (n_pages, 2, H, page, D) if pool else (2, n_pages, page, H, D)
    both = torch.empty(shape, dtype=torch.uint8, device="cuda")
    views = [both[:, s].transpose(1, 2) if pool else both[s] for s in (0, 1)]
    scales = torch.empty(n_pages, 2, H, nb, device="cuda")
    step = max(1, (1 << 26) // (page * H * D))
    for s in (0, 1):
        for p0 in range(0, n_pages, step):
            n = min(step, n_pages - p0)
            x = torch.randn(n, nb, blk, H, D, generator=gen, device="cuda")
            x *= torch.exp(0.5 * torch.randn(n, nb, 1, H, 1, generator=gen, device="cuda"))
            x *= 1 + 7 * (torch.rand(n, nb, 1, H, D, generator=gen, device="cuda") < 0.01)  # channels that stand out
            amax = x.abs().amax((2, 4))
            sc = pow2_scale(amax, c["fmt"]) if pow2 else amax / top
            x = (x / sc[:, :, None, :, None]).clamp(-top, top).to(kind).view(torch.uint8)
            views[s][p0:p0 + n] = x.reshape(n, page, H, D)
            scales[p0:p0 + n, s] = sc.transpose(1, 2)
    return views[0], views[1], scales


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    pairs = lengths(c)
    q, H, D, blk, B, op = c["q"], c["Hkv"], c["D"], c["block"], c["B"], c["op"]
    top = max(L for L, _ in pairs)
    st = {"case": dict(c), "seq": torch.tensor(pairs, dtype=torch.int32, device="cuda"), "top": top}
    if op == "select":
        n = blocks(top, blk)
        x = 3 * torch.randn(B, 1, H, n, generator=gen, device="cuda") + torch.randn(B, q, H, n, generator=gen, device="cuda")
        st["scores"] = (x * 8).round() / 8 if c["k"] % 2 else x  # coarse scores: many ties
        st["ids"] = torch.full((B, q, H, c["k"]), -7, dtype=torch.int32, device="cuda")
        return st
    per = [blocks(L, c["page"]) for L, _ in pairs]
    n_pages = sum(per) + 3
    order = torch.randperm(n_pages, generator=gen, device="cuda").int()
    table = torch.full((B, max(per)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    st["table"] = table
    if op == "append":
        st["k_cache"], st["v_cache"], st["scales"] = cache(c, n_pages, gen, True)
        kind = torch.bfloat16 if c["dtype"] == "bf16" else torch.float16
        for name in ("k_new", "v_new"):
            x = torch.randn(B, q, H, D, generator=gen, device="cuda")
            x *= torch.exp(0.5 * torch.randn(B, q, H, 1, generator=gen, device="cuda"))
            st[name] = x.to(kind)
        st["bounds"] = torch.zeros(n_pages, H, c["page"] // blk, 2, D, dtype=torch.uint8, device="cuda") if c["bounds"] else None
        return st
    st["q"] = torch.randn(B, q, c["Hq"], D, generator=gen, device="cuda").half()
    if op == "scores":
        nb, (kind, big, _) = c["page"] // blk, FP8[c["fmt"]]
        x = torch.randn(n_pages, H, nb, 2, D, generator=gen, device="cuda") * 100
        x = torch.stack([x.amin(3) - 50, x.amax(3) + 50], 3).clamp(-big, big)
        st["bounds"] = x.to(kind).view(torch.uint8)
        st["scales"] = torch.exp(torch.randn(n_pages, 2, H, nb, generator=gen, device="cuda") * 0.5 - 5)
        st["scores"] = torch.zeros(B, q, H, blocks(top, blk), device="cuda")
        return st
    st["k_cache"], st["v_cache"], st["scales"] = cache(c, n_pages, gen, False)
    st["out"] = torch.zeros(B, q, c["Hq"], D, dtype=torch.float16, device="cuda")
    if op == "sparse":
        # every query: the last block, blocks that all queries share, and `apart` blocks of its own
        k, apart = c["k"], c["apart"]
        ids = torch.full((B, q, H, k), -1, dtype=torch.int32, device="cuda")
        for b, (L, n) in enumerate(pairs):
            last = blocks(L, blk) - 1
            mix = torch.rand(H, last, generator=gen, device="cuda").argsort(-1).int()
            same = mix[:, :k - 1 - apart]
            for i in range(n):
                mine = mix[:, k - 1 - apart + i * apart:k - 1 - apart + (i + 1) * apart]
                tail = torch.full((H, 1), last, dtype=torch.int32, device="cuda")
                ids[b, i] = torch.cat([same, mine, tail], -1).sort(-1).values[:, :k]
        st["ids"] = ids
    return st


# ---------------------------------------------------------------------------- a pass


def run(st):
    return globals()[("own_" if own else "plain_") + st["case"]["op"]](st)


def fp8(t, c):
    return t.view(FP8[c["fmt"]][0])


def plain_append(st):
    c = st["case"]
    kind, top, _ = FP8[c["fmt"]]
    page, blk, H, D, B, Q = c["page"], c["block"], c["Hkv"], c["D"], c["B"], c["q"]
    L, n = st["seq"][:, 0].long(), st["seq"][:, 1].long()
    nt = Q // blk + 2  # blocks that a sequence's new tokens can touch
    first = (L - n) // blk
    lb = first[:, None] + torch.arange(nt, device="cuda")  # [B][nt] logical block
    live = lb * blk < L[:, None]
    pg = st["table"].long().gather(1, (lb * blk // page).clamp(max=st["table"].shape[1] - 1))
    pg = torch.where(live, pg, 0)
    sub = (lb * blk % page) // blk
    tok = lb[:, :, None] * blk + torch.arange(blk, device="cuda")  # [B][nt][blk]
    is_new = (tok >= (L - n)[:, None, None]) & (tok < L[:, None, None])
    is_old = (tok < (L - n)[:, None, None])
    kept = is_new | is_old
    slot = tok % page
    src = (tok - (L - n)[:, None, None]).clamp(0, Q - 1)
    rows = torch.arange(B, device="cuda")[:, None, None]
    has_old = is_old.any(-1)
    for which, new, dst in ((0, st["k_new"], st["k_cache"]), (1, st["v_new"], st["v_cache"])):
        x = torch.where(is_new[..., None, None], new[rows, src].float(), 0)  # [B][nt][blk][H][D]
        old_s = st["scales"][pg, which, :, sub]  # [B][nt][H]
        need = pow2_scale(x.abs().amax((2, 4)), c["fmt"])
        s = torch.where(has_old[..., None], torch.maximum(old_s, need), need)
        codes = dst[pg[..., None], slot]
        was = codes.view(kind).float() * (old_s / s)[:, :, None, :, None]
        y = torch.where(is_new[..., None, None], x / s[:, :, None, :, None], was).clamp(-top, top)
        y = torch.where(kept[..., None, None], y, 0).to(kind)
        put = kept & live[..., None]
        dst[pg[..., None].expand_as(tok)[put], slot[put]] = y.view(torch.uint8)[put]
        st["scales"][pg[live], which, :, sub[live]] = s[live]
        if which == 0 and st["bounds"] is not None:
            v = y.float()
            none = ~kept[..., None, None]
            lo = torch.where(none, math.inf, v).amin(2)
            hi = torch.where(none, NEG, v).amax(2)
            both = torch.stack([lo, hi], 3).to(kind).view(torch.uint8)  # [B][nt][H][2][D]
            st["bounds"][pg[live], :, sub[live]] = both[live]
    return outputs_append(st)


def outputs_append(st):
    c = st["case"]
    out = {"k_cache": fp8(st["k_cache"], c), "v_cache": fp8(st["v_cache"], c), "scales": st["scales"]}
    if st["bounds"] is not None:
        out["bounds"] = fp8(st["bounds"], c)
    return out


def plain_attention(st, K, V, ks, vs, pos, ok):
    """softmax(q K^T) V: K, V [B][i or 1][t][H][D], scales and positions and truth of the same rows, in 32 bits."""
    c = st["case"]
    B, Q, H, G, D = c["B"], c["q"], c["Hkv"], c["Hq"] // c["Hkv"], c["D"]
    K = K.float() * ks[..., None]
    V = V.float() * vs[..., None]
    T = K.shape[1]  # Q where every query has keys of its own, else 1
    qq = st["q"].float().view(B, T, Q // T, H, G, D).transpose(2, 3).reshape(B, T, H, Q // T * G, D)
    i = torch.arange(Q, device="cuda")
    L, n = st["seq"][:, 0, None], st["seq"][:, 1, None]
    see = (L - n + i)[:, :, None, None]  # last position that query i sees
    mask = ok & (pos <= see) & (i < n)[:, :, None, None]  # [B][Q][t][H]
    z = torch.matmul(qq, K.permute(0, 1, 3, 4, 2)) / math.sqrt(D)
    z = z.view(B, T, H, Q // T, G, -1).transpose(2, 3).reshape(B, Q, H, G, -1)
    z = z.masked_fill(~mask.permute(0, 1, 3, 2)[:, :, :, None], NEG)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(m == NEG, 0, m))
    weights = p.view(B, T, Q // T, H, G, -1).transpose(2, 3).reshape(B, T, H, Q // T * G, -1)
    o = torch.matmul(weights, V.permute(0, 1, 3, 2, 4))
    o = o.view(B, T, H, Q // T, G, D).transpose(2, 3).reshape(B, Q, H, G, D)
    o = o / p.sum(-1, keepdim=True).clamp_min(1e-38)
    return o.reshape(B, Q, H * G, D).half()


def plain_attend(st):
    c = st["case"]
    t = torch.arange(st["top"], device="cuda")
    lp = t // c["page"]
    pg = st["table"].long()[:, lp].clamp_min(0)  # [B][t]
    slot = t % c["page"]
    K = fp8(st["k_cache"][pg, slot], c)[:, None]
    V = fp8(st["v_cache"][pg, slot], c)[:, None]
    sub = slot // c["block"]
    ks, vs = st["scales"][pg, 0, :, sub][:, None], st["scales"][pg, 1, :, sub][:, None]
    pos = t[None, None, :, None]
    st["out"].copy_(plain_attention(st, K, V, ks, vs, pos, pos < st["seq"][:, 0, None, None, None]))
    return st["out"]


def plain_scores(st):
    c = st["case"]
    B, Q, H, G, D, blk = c["B"], c["q"], c["Hkv"], c["Hq"] // c["Hkv"], c["D"], c["block"]
    j = torch.arange(st["scores"].shape[-1], device="cuda")
    pg = st["table"].long()[:, j * blk // c["page"]].clamp_min(0)
    sub = j * blk % c["page"] // blk
    bd = fp8(st["bounds"][pg, :, sub], c).float()  # [B][n][H][2][D]
    sc = st["scales"][pg, 0, :, sub]  # [B][n][H]
    qq = st["q"].float().view(B, Q, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, Q * G, D)
    lo, hi = bd[:, :, :, 0].permute(0, 2, 3, 1), bd[:, :, :, 1].permute(0, 2, 3, 1)  # [B][H][D][n]
    u = torch.matmul(qq.clamp_min(0), hi) + torch.matmul(qq.clamp_max(0), lo)
    u = u.view(B, H, Q, G, -1).amax(3).permute(0, 2, 1, 3) * sc.permute(0, 2, 1)[:, None] / math.sqrt(D)
    i = torch.arange(Q, device="cuda")
    L, n = st["seq"][:, 0, None], st["seq"][:, 1, None]
    see = (L - n + i)[:, :, None, None]
    u = torch.where(j * blk <= see, u, NEG)
    write = (j * blk < L[:, :, None, None]) & (i < n)[:, :, None, None]
    st["scores"].copy_(torch.where(write, u, st["scores"]))
    return st["scores"]


def plain_select(st):
    c = st["case"]
    x = st["scores"]
    i = torch.arange(c["q"], device="cuda")
    L, n = st["seq"][:, 0, None].long(), st["seq"][:, 1, None].long()
    vis = ((L - n + i) // c["block"] + 1)[:, :, None, None]  # blocks that query i sees
    j = torch.arange(x.shape[-1], device="cuda").expand(x.shape)
    tier = torch.where((j < c["sink"]) | (j >= vis - c["local"]), 2, 1)
    tier = torch.where((j < vis) & (i < n)[:, :, None, None], tier, 0)
    order = torch.where(x != x, NEG, x).sort(stable=True, dim=-1, descending=True).indices
    order = order.gather(-1, tier.gather(-1, order).sort(stable=True, dim=-1, descending=True).indices)
    pick = order[..., :c["k"]]
    far = x.shape[-1]
    ids = torch.where(tier.gather(-1, pick) > 0, pick, far).sort(-1).values
    ids = torch.where(ids == far, -1, ids).int()
    st["ids"].fill_(-1)
    st["ids"][..., :ids.shape[-1]] = ids
    return st["ids"]


def plain_sparse(st):
    c = st["case"]
    blk, B, Q, H = c["block"], c["B"], c["q"], c["Hkv"]
    ids = st["ids"].long().transpose(2, 3)  # [B][Q][k][H]
    t = torch.arange(blk, device="cuda")
    pos = (ids[:, :, :, None] * blk + t[:, None]).reshape(B, Q, -1, H)  # [B][Q][k * block][H]
    ok = (pos >= 0) & (pos < st["seq"][:, 0, None, None, None])
    at = pos.clamp(0, st["table"].shape[1] * c["page"] - 1)
    pg = st["table"].long()[torch.arange(B, device="cuda")[:, None, None, None], at // c["page"]].clamp_min(0)
    slot, h = at % c["page"], torch.arange(H, device="cuda")
    K, V = fp8(st["k_cache"][pg, slot, h], c), fp8(st["v_cache"][pg, slot, h], c)
    ks, vs = st["scales"][pg, 0, h, slot // blk], st["scales"][pg, 1, h, slot // blk]
    st["out"].copy_(plain_attention(st, K, V, ks, vs, pos, ok))
    return st["out"]


# ---------------------------------------------------------------------------- the package's calls


def own_append(st):
    import fp8_paged_attention_e4m3_gb300 as vae4
    vae4.verify_attn_e4m3_append(st["k_new"], st["v_new"], st["k_cache"], st["v_cache"], st["table"], st["seq"],
                                 st["scales"], k_bounds=st["bounds"], flags=own_flags(vae4, st))
    return outputs_append(st)


def own_flags(vae4, st):
    return vae4.FLAG_KV_E5M2 if st["case"]["fmt"] == "e5m2" else 0


def own_attend(st):
    import fp8_paged_attention_e4m3_gb300 as vae4
    c = st["case"]
    if "ws" not in st:  # a program keeps its workspace from step to step
        st["ws"] = vae4.alloc_workspace(c["B"], c["Hq"], c["Hkv"], c["q"], c["D"], st["top"])
    return vae4.verify_attn_e4m3_block_scaled(st["q"], st["k_cache"], st["v_cache"], st["table"], st["seq"], st["scales"],
                                              st["out"], st["ws"], max_seq_len=st["top"], flags=own_flags(vae4, st))


def own_scores(st):
    import fp8_paged_attention_e4m3_gb300 as vae4
    return vae4.verify_attn_e4m3_block_scores(st["q"], st["bounds"], st["table"], st["seq"], st["scales"], st["scores"],
                                              block_tokens=st["case"]["block"], flags=own_flags(vae4, st))


def own_select(st):
    import fp8_paged_attention_e4m3_gb300 as vae4
    c = st["case"]
    return vae4.verify_attn_e4m3_select_blocks(st["scores"], st["seq"], st["ids"], block_tokens=c["block"],
                                               sink_blocks=c["sink"], local_blocks=c["local"])


def own_sparse(st):
    import fp8_paged_attention_e4m3_gb300 as vae4
    c = st["case"]
    if "ws" not in st:
        st["ws"] = vae4.alloc_sparse_workspace(c["B"], c["Hq"], c["Hkv"], c["q"], c["D"], st["top"], c["block"], c["k"])
    return vae4.verify_attn_e4m3_sparse(st["q"], st["k_cache"], st["v_cache"], st["table"], st["seq"], st["scales"], st["ids"],
                                        st["out"], st["ws"], max_seq_len=st["top"], flags=own_flags(vae4, st))


# ---------------------------------------------------------------------------- 64 bits, from the definitions


def exact(c, seed):
    return globals()["exact_" + c["op"]](c, prepare(c, seed))


def pages_of(st, b, L, page):
    return st["table"][b, :blocks(L, page)].long()


def values(st, c, which, b, L):
    """The L values [L][H][D] of sequence b that K (0) or V (1) stands for."""
    raw = (st["k_cache"], st["v_cache"])[which][pages_of(st, b, L, c["page"])]  # [pages][page][H][D]
    x = raw.contiguous().view(FP8[c["fmt"]][0]).double()
    s = st["scales"][pages_of(st, b, L, c["page"]), which].double()  # [pages][H][nb]
    x = x * s.repeat_interleave(c["block"], 2).transpose(1, 2)[..., None]
    return x.flatten(0, 1)[:L]


def exact_attention(c, st, picked):
    """picked(b, i, h, L): truth for each of the L keys."""
    G, D = c["Hq"] // c["Hkv"], c["D"]
    out = torch.zeros(c["B"], c["q"], c["Hq"], D, dtype=torch.float64, device="cuda")
    for b, (L, n) in enumerate(lengths(c)):
        K, V = values(st, c, 0, b, L), values(st, c, 1, b, L)
        for i in range(n):
            seen = L - n + i + 1
            for h in range(c["Hkv"]):
                keep = picked(b, i, h, seen)
                if not keep.numel():
                    continue
                z = st["q"][b, i, h * G:(h + 1) * G].double() @ K[keep, h].T / math.sqrt(D)
                out[b, i, h * G:(h + 1) * G] = torch.softmax(z, -1) @ V[keep, h]
    return out


def exact_attend(c, st):
    return exact_attention(c, st, lambda b, i, h, seen: torch.arange(seen, device="cuda"))


def exact_sparse(c, st):
    def picked(b, i, h, seen):
        ids = st["ids"][b, i, h]
        keys = (ids[ids >= 0].long()[:, None] * c["block"] + torch.arange(c["block"], device="cuda")).flatten()
        return keys[keys < seen]
    return exact_attention(c, st, picked)


def exact_scores(c, st):
    out = st["scores"].double()
    G, D, blk = c["Hq"] // c["Hkv"], c["D"], c["block"]
    for b, (L, n) in enumerate(lengths(c)):
        nb = blocks(L, blk)
        bd = st["bounds"][pages_of(st, b, L, c["page"])].view(FP8[c["fmt"]][0]).double()  # [pages][H][nb][2][D]
        bd = bd.transpose(0, 1).flatten(1, 2)[:, :nb]
        s = st["scales"][pages_of(st, b, L, c["page"]), 0].double().transpose(0, 1).flatten(1, 2)[:, :nb]
        for i in range(n):
            qi = st["q"][b, i].double().view(c["Hkv"], G, D)
            hi = torch.einsum("hgd,hnd->hgn", qi.clamp_min(0), bd[:, :, 1]) + torch.einsum("hgd,hnd->hgn", qi.clamp_max(0), bd[:, :, 0])
            u = hi.amax(1) * s / math.sqrt(D)
            u[:, (L - n + i) // blk + 1:] = NEG
            out[b, i, :, :nb] = u
    return out


def exact_select(c, st):
    return None  # whole numbers


def exact_append(c, st):
    kind, top, lead = FP8[c["fmt"]]
    page, blk = c["page"], c["block"]
    kc, vc, sc = st["k_cache"].clone(), st["v_cache"].clone(), st["scales"].clone()
    bd = st["bounds"].clone() if st["bounds"] is not None else None
    work_on = {}
    for b, (L, n) in enumerate(lengths(c)):
        for j in range((L - n) // blk, blocks(L, blk)):
            if len(work_on) > 4000:
                return None  # a long prompt: one block after another takes too long here
            t0, a, z = j * blk, max(j * blk, L - n), min((j + 1) * blk, L)
            work_on[b, j] = (st["table"][b, t0 // page], t0 % page, a - t0, z - t0, a - (L - n), z - (L - n))
    for (b, j), (pg, slot, a, z, x0, x1) in work_on.items():
        for which, new, dst in ((0, st["k_new"], kc), (1, st["v_new"], vc)):
            x = new[b, x0:x1].double()  # [t][H][D]
            amax = x.abs().amax((0, 2))
            e = torch.floor(torch.log2(amax.clamp_min(1e-300)))
            e = e - lead + (amax > top * torch.exp2(e - lead)).double()
            s = torch.exp2(torch.where(amax > 0, e, -30.0).clamp(-30, 30))
            old = dst[pg, slot:slot + a].view(kind).double()
            if a:
                was = sc[pg, which, :, slot // blk].double()
                s = torch.maximum(s, was)
                old = old * (was / s)[None, :, None]
            y = torch.cat([old, x / s[None, :, None]]).clamp(-top, top).float().to(kind)
            dst[pg, slot:slot + z] = y.view(torch.uint8)
            sc[pg, which, :, slot // blk] = s.float()
            if bd is not None and which == 0:
                v = y.double()
                bd[pg, :, slot // blk] = torch.stack([v.amin(0), v.amax(0)], 1).float().to(kind).view(torch.uint8)
    out = {"k_cache": kc.view(kind).double(), "v_cache": vc.view(kind).double(), "scales": sc.double()}
    if bd is not None:
        out["bounds"] = bd.view(kind).double()
    return out
