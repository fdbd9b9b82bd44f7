"""The operators of the 8-bit paged cache, as they are measured.

Five operators, each in a plain form (elementary torch operations, 32 bits or
more, rounded once) and, with ``own``, as the library's call:

* append: new tokens' K and V enter a paged e4m3 cache with one scale per page
  and KV head;
* attn: attention over the selected blocks of that cache;
* scored: the same with capped scores, a distance bias and per-query windows
  (documents, a bidirectional prefix);
* weight: the attention weight each block received, accumulated per sequence;
* evict: the blocks with the least accumulated weight leave the cache.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
MIN_EXP = -60  # smallest scale 2^-60
LOG2E = 1.4426950408889634


def listed():
    return [
        # one new token of 32 sequences at 32K context: the write of a serving step
        dict(name="append_decode", op="append", B=32, T=1, ctx=32768, H_kv=1, hd=128, bs=64, dtype="bf16", ragged=False),
        # four ragged prompts of up to 8191 tokens behind a cached turn, 8 KV heads: the write of a prompt
        dict(name="append_prompt", op="append", B=4, T=8191, ctx=1003, H_kv=8, hd=128, bs=64, dtype="bf16", ragged=True),
        # one token at 1M context, 16 blocks of 128: the smallest attention call, where latency counts
        dict(name="attn_1m_decode", op="attn", B=1, S=1, ctx=1048576, topk=16, H_kv=1, G=16, hd=128, bs=128, dtype="bf16", mass=True),
        # 32 sequences at up to 32K, 32 blocks of 64: the ordinary serving step, with the blocks' weights for eviction
        dict(name="attn_decode", op="attn", B=32, S=1, ctx=32768, topk=32, H_kv=1, G=16, hd=128, bs=64, dtype="bf16", mass=True),
        # an 8K prompt, 32 blocks per query: the largest call, compute-bound
        dict(name="attn_prefill", op="attn", B=1, S=8192, ctx=8192, topk=32, H_kv=1, G=16, hd=128, bs=64, dtype="bf16", mass=False),
        # the small fp32 configuration used for parity: blocks of 16 tokens, head size 64
        dict(name="attn_tiny_f32", op="attn", B=1, S=256, ctx=256, topk=4, H_kv=4, G=1, hd=64, bs=16, dtype="f32", mass=False),
        # long decode (8 sequences at 256K, 64 blocks, 32 heads on 2) with capped scores and a distance bias
        dict(name="scored_long_decode", op="scored", B=8, S=1, ctx=262144, topk=64, H_kv=2, G=16, hd=128, bs=64, dtype="bf16", mass=True, cap=50.0, slopes=True, window="none", span=0),
        # packed documents of 1500 tokens in two 4096-token rows: capped scores behind a document mask
        dict(name="scored_packed_prefill", op="scored", B=2, S=4096, ctx=4096, topk=16, H_kv=2, G=8, hd=128, bs=64, dtype="bf16", mass=False, cap=30.0, slopes=False, window="docs", span=1500),
        # accumulating the weights of a serving step (32 sequences of 512 blocks)
        dict(name="weight_decode", op="weight", B=32, S=1, topk=32, H_kv=1, NB=512, decay=0.95),
        # accumulating the weights of an 8K prompt
        dict(name="weight_prompt", op="weight", B=1, S=8192, topk=32, H_kv=1, NB=128, decay=1.0),
        # trimming 32 sequences of 512 blocks to half
        dict(name="evict_decode", op="evict", B=32, NB=512, bs=64, budget=256, sink=1, recent=4, levels=0),
        # trimming 8 sequences of up to 16384 blocks, weights with many ties
        dict(name="evict_long", op="evict", B=8, NB=16384, bs=64, budget=9001, sink=4, recent=32, levels=1000),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "scored", "scored", "weight", "evict"])
    if op == "append":
        H_kv = rng.choice([1, 2, 4, 8])
        T = 1 if rng.random() < 0.3 else _log_int(rng, 2, 8192)
        B = min(_log_int(rng, 1, 64), max(1, 4 * 8191 * 4 // (T * H_kv)))
        return dict(op="append", B=B, T=T, ctx=_log_int(rng, 1, 8192), H_kv=H_kv, hd=rng.choice([64, 96, 128, 128]), bs=rng.choice([16, 48, 64, 64, 128]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), ragged=rng.random() < 0.5)
    if op in ("attn", "scored"):
        f32 = rng.random() < 0.15
        if f32:
            c = dict(op=op, B=rng.randint(1, 3), S=_log_int(rng, 1, 200), H_kv=rng.choice([1, 2, 4]), G=rng.randint(1, 8), hd=rng.choice([32, 64, 96]), bs=rng.choice([8, 16, 48]), dtype="f32")
            c["topk"] = rng.randint(1, 8)
            c["ctx"] = c["S"] + _log_int(rng, 1, 400)
            c["mass"] = False
        else:
            decode = rng.random() < 0.5
            H_kv, G, bs = rng.choice([1, 2, 4]), rng.choice([1, 3, 4, 8, 8, 16, 16]), rng.choice([64, 64, 128])
            S = rng.randint(1, 4) if decode else _log_int(rng, 16, 4096)
            B = _log_int(rng, 1, 64) if decode else rng.randint(1, 3)
            ctx = min(S + _log_int(rng, 1, 131072 if decode else 16384), 4194304 // (B * H_kv))
            ctx = max(ctx, S)
            topk = _log_int(rng, 1, 128)
            while topk > 1 and B * S * H_kv * topk * bs * max(G, 16) > (1 << 23 if decode else 16 * 8192 * 1780):
                topk //= 2
            c = dict(op=op, B=B, S=S, ctx=ctx, topk=topk, H_kv=H_kv, G=G, hd=128, bs=bs, dtype="bf16", mass=decode and rng.random() < 0.7)
        if op == "scored":
            c["cap"] = rng.choice([0.0, 20.0, 50.0])
            c["slopes"] = rng.random() < 0.5
            c["window"] = rng.choice(["none", "docs", "prefix"])
            c["span"] = 0 if c["window"] == "none" else _log_int(rng, 16, max(17, c["ctx"]))
        return c
    if op == "weight":
        B, H_kv, topk, NB = _log_int(rng, 1, 32), rng.choice([1, 2, 4]), _log_int(rng, 1, 128), _log_int(rng, 8, 16384)
        S = 1 if rng.random() < 0.4 else _log_int(rng, 2, 8192)
        S = max(1, min(S, 8192 * 64 // (B * H_kv * topk)))
        return dict(op="weight", B=B, S=S, topk=min(topk, NB), H_kv=H_kv, NB=NB, decay=rng.choice([1.0, 0.9]))
    NB = _log_int(rng, 8, 16384)
    B = min(_log_int(rng, 1, 64), max(1, 8 * 16384 // NB))
    budget = rng.randint(2, NB)
    sink = rng.randint(0, min(4, budget - 1))
    return dict(op="evict", B=B, NB=NB, bs=rng.choice([64, 128]), budget=budget, sink=sink, recent=rng.randint(1, min(64, budget - sink)), levels=rng.choice([0, 3, 1000]))


# ---------------------------------------------------------------- sizes of a case

def _lens(c):
    """Context length of each sequence: from `ctx` down to half of it."""
    return [c["ctx"] - (b * (c["ctx"] - c["S"])) // (2 * c["B"]) for b in range(c["B"])]


def _counts(c):
    """New tokens of each sequence of an append."""
    return [c["T"] - (b * c["T"]) // (c["B"] + 1) if c["ragged"] else c["T"] for b in range(c["B"])]


def _starts(c):
    return [max(0, c["ctx"] - 1 - 37 * b) for b in range(c["B"])]


def _windows(c, p, n):
    """First and last position a query at position p of an n-token context may see."""
    if c.get("window", "none") == "docs":
        return (p // c["span"]) * c["span"], min(p, n - 1)
    if c.get("window", "none") == "prefix":
        return 0, min(max(p, c["span"] - 1), n - 1)
    return 0, min(p, n - 1)


def work(c):
    if c["op"] == "append":
        new = sum(_counts(c)) * c["H_kv"] * c["hd"] * 2
        return {"bytes": new * ((2 if c["dtype"] == "bf16" else 4) + 1), "flops": 4 * new}
    if c["op"] in ("attn", "scored"):
        bs, picked, seen = c["bs"], 0, 0
        for n in _lens(c):
            got, blocks = 0, 0
            for s in range(c["S"]):
                lo, hi = _windows(c, n - c["S"] + s, n)
                k = min(c["topk"], hi // bs - lo // bs + 1)
                got += min(k * bs, hi - lo + 1)
                blocks += k
            picked += got
            seen += min(got, n)
        e = 2 if c["dtype"] == "bf16" else 4
        rows = c["B"] * c["S"]
        return {"bytes": seen * c["H_kv"] * c["hd"] * 2 + 2 * rows * c["H_kv"] * c["G"] * c["hd"] * e + 4 * rows * c["topk"] * (1 + (c["H_kv"] if c["mass"] else 0)),
                "flops": 4 * picked * c["H_kv"] * c["G"] * c["hd"]}
    if c["op"] == "weight":
        n = c["B"] * c["S"] * c["topk"]
        return {"bytes": 4 * n * (1 + c["H_kv"]) + 8 * c["B"] * c["NB"], "flops": n * c["H_kv"]}
    return {"bytes": 16 * c["B"] * c["NB"], "flops": c["B"] * c["NB"]}


# ---------------------------------------------------------------- inputs

def _cache(c, gen, pages, lens_total):
    """Pools of e4m3 values with a power-of-two scale per page and head; pages
    no sequence holds, and slots behind the last token, hold NaN codes."""
    dev = "cuda"
    out = []
    for spread in (1.0, 2.0):
        shape = (pages, c["H_kv"], c["bs"], c["hd"])
        x = torch.randn(shape, generator=gen, device=dev)
        x *= torch.exp2((torch.rand(pages, c["H_kv"], 1, 1, generator=gen, device=dev) - 0.5) * spread)
        amax = x.abs().amax(dim=(2, 3))
        scale = torch.exp2(torch.ceil(torch.log2(amax / E4M3_MAX)))
        codes = (x / scale[:, :, None, None]).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        del x
        out += [codes, scale]
    return out[0], out[2], out[1], out[3]


def _blank(pool, scale, table, lens, bs):
    """NaN codes wherever no token is stored."""
    raw = pool.view(torch.uint8)
    used = torch.zeros(pool.shape[0], dtype=torch.bool, device=pool.device)
    for b, n in enumerate(lens):
        nb = -(-n // bs)
        used[table[b, :nb].long()] = True
        if n % bs:
            raw[int(table[b, nb - 1]), :, n % bs:] = 0x7F
    raw[~used] = 0x7F
    scale[~used] = 0.0


def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dev = "cuda"
    st = dict(c)
    if c["op"] == "weight":
        B, S, topk, NB = c["B"], c["S"], c["topk"], c["NB"]
        rows = max(1, (1 << 26) // NB)
        ids = torch.empty(B * S, topk, dtype=torch.int32, device=dev)
        for r in range(0, B * S, rows):
            ids[r:r + rows] = torch.rand(min(rows, B * S - r), NB, generator=gen, device=dev).topk(topk, dim=1).indices.to(torch.int32)
        ids[torch.rand(B * S, topk, generator=gen, device=dev) < 0.02] = -1
        mass = torch.rand(B, S, c["H_kv"], topk, generator=gen, device=dev) ** 4
        mass *= 16.0 / mass.sum(dim=-1, keepdim=True)
        st.update(ids=ids.reshape(B, S, topk), mass=mass, weight=torch.rand(B, NB, generator=gen, device=dev))
        if own:
            import long_context_indexer_b200 as lci
            st["call"] = lci.prepare_block_weight_update(st["weight"], st["ids"], st["mass"], decay=c["decay"])
        return st
    if c["op"] == "evict":
        B, NB = c["B"], c["NB"]
        weight = torch.rand(B, NB, generator=gen, device=dev) ** 3 * 10
        if c["levels"]:
            weight = torch.floor(weight * c["levels"] / 10)
        table = torch.randperm(B * NB + 5, generator=gen, device=dev)[: B * NB].reshape(B, NB).to(torch.int32)
        ctx = torch.tensor([(NB - b * NB // (3 * B)) * c["bs"] - 5 for b in range(B)], dtype=torch.int32, device=dev)
        st.update(weight=weight, table=table, ctx_len=ctx)
        if own:
            import long_context_indexer_b200 as lci
            st["bt"] = lci.BlockTable(table, B * NB + 5, c["bs"], 1, 128, torch.float8_e4m3fn)
            st["call"] = lci.prepare_cache_evict(st["bt"], ctx, weight, c["budget"], sink=c["sink"], recent=c["recent"])
        return st
    B, bs = c["B"], c["bs"]
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    if c["op"] == "append":
        starts, counts = _starts(c), _counts(c)
        lens = [s + n for s, n in zip(starts, counts)]
        NB = -(-max(s + c["T"] for s in starts) // bs)
    else:
        lens = _lens(c)
        NB = -(-c["ctx"] // bs)
    pages = B * NB + 3
    table = torch.randperm(pages, generator=gen, device=dev)[: B * NB].reshape(B, NB).to(torch.int32).contiguous()
    k, v, ks, vs = _cache(c, gen, pages, sum(lens))
    for pool, scale in ((k, ks), (v, vs)):
        _blank(pool, scale, table, starts if c["op"] == "append" else lens, bs)
    st.update(k=k, v=v, ks=ks, vs=vs, table=table)
    if c["op"] == "append":
        shape = (B, c["T"], c["H_kv"], c["hd"])
        # a few outlying tokens, so that scales grow and stored tokens are re-rounded
        grow = 1 + 7 * (torch.rand(B, c["T"], c["H_kv"], 1, generator=gen, device=dev) < 0.05).float()
        st["k_new"] = (torch.randn(shape, generator=gen, device=dev) * grow).to(dt)
        st["v_new"] = (torch.randn(shape, generator=gen, device=dev) * grow).to(dt)
        st["start"] = torch.tensor(starts, dtype=torch.int32, device=dev)
        st["count"] = torch.tensor(counts, dtype=torch.int32, device=dev) if c["ragged"] else None
        if own:
            import long_context_indexer_b200 as lci
            cache = lci.Q8Cache.wrap(k, v, ks, vs)
            st["bt"] = lci.create_block_table(table, k)
            st["call"] = lci.prepare_kv_append_q8(cache, st["bt"], st["k_new"], st["v_new"], st["start"], count=st["count"])
        return st
    S, topk = c["S"], c["topk"]
    st["q"] = torch.randn(B, S, c["H_kv"] * c["G"], c["hd"], generator=gen, device=dev).to(dt)
    st["ctx_len"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    st["q_start"] = st["ctx_len"] - S
    p = st["q_start"][:, None] + torch.arange(S, device=dev, dtype=torch.int32)[None]
    st["first"] = st["last"] = st["slopes"] = None
    lo, hi = torch.zeros_like(p), p
    if c["op"] == "scored":
        if c["window"] == "docs":
            st["first"] = lo = (p // c["span"]) * c["span"]
        if c["window"] == "prefix":
            st["last"] = hi = p.clamp(min=c["span"] - 1)
        if c["slopes"]:
            Hq = c["H_kv"] * c["G"]
            st["slopes"] = torch.exp2(-8.0 * (torch.arange(Hq, device=dev) + 1) / Hq).float()
    hi = torch.minimum(hi, st["ctx_len"][:, None] - 1)
    # the selected blocks of each query, in no order of position, -1 where fewer are visible
    ids = torch.full((B * S, topk), -1, dtype=torch.int32, device=dev)
    jlo, jhi = (lo // bs).reshape(-1, 1), (hi // bs).reshape(-1, 1)
    j = torch.arange(NB, device=dev)[None]
    k_eff, rows = min(topk, NB), max(1, (1 << 26) // NB)
    for r in range(0, B * S, rows):
        x = torch.rand(min(rows, B * S - r), NB, generator=gen, device=dev)
        x = torch.where((j >= jlo[r:r + rows]) & (j <= jhi[r:r + rows]), x, -1.0)
        best = x.topk(k_eff, dim=1)
        ids[r:r + rows, :k_eff] = torch.where(best.values >= 0, best.indices, -1).to(torch.int32)
    st["ids"] = ids.reshape(B, S, topk)
    if own:
        import long_context_indexer_b200 as lci
        cache = lci.Q8Cache.wrap(k, v, ks, vs)
        st["bt"] = lci.create_block_table(table, k)
        st["call"] = lci.prepare_sparse_attn_q8(st["q"], cache, st["bt"], st["ids"], st["ctx_len"], st["q_start"], cap=c.get("cap", 0.0), slopes=st["slopes"],
                                                first=st["first"], last=st["last"], lse=True, mass=c["mass"])
    return st


# ---------------------------------------------------------------- plain forms

def _pow2_scale(amax):
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8)  # smallest e with amax <= 448 * 2^e (448 = 0.875 * 2^9)
    e = torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp(min=MIN_EXP)
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _append(st):
    B, T, H, hd, bs = st["B"], st["T"], st["H_kv"], st["hd"], st["bs"]
    dev = st["table"].device
    t = torch.arange(T, device=dev)
    count = st["count"] if st["count"] is not None else torch.full((B,), T, device=dev)
    b, t = torch.nonzero(t[None] < count[:, None], as_tuple=True)
    pos = st["start"].long()[b] + t
    page, slot = st["table"][b, pos // bs].long(), pos % bs
    part = st["start"].long() % bs
    part = torch.where(count > 0, part, torch.zeros_like(part))
    head = st["table"][torch.arange(B, device=dev), (st["start"].long() // bs).clamp(max=st["table"].shape[1] - 1)].long()
    for new, pool, scale in ((st["k_new"], st["k"], st["ks"]), (st["v_new"], st["v"], st["vs"])):
        x = new[b, t].float()
        a = torch.where(x.isfinite(), x.abs(), torch.zeros_like(x)).amax(dim=-1)
        amax = torch.zeros_like(scale).scatter_reduce_(0, page[:, None].expand(-1, H), a, "amax")
        held = torch.zeros(scale.shape[0], dtype=torch.bool, device=dev)
        held[head[part > 0]] = True
        old = torch.where(held[:, None], scale, torch.zeros_like(scale))
        fresh = torch.maximum(old, _pow2_scale(amax))
        raw = pool.view(torch.uint8)
        # stored tokens of a page that gets more: to the new scale
        hp, hn = head[part > 0], part[part > 0]
        ratio = (old[hp] / fresh[hp])[:, :, None, None]
        again = (raw[hp].view(torch.float8_e4m3fn).float() * ratio).to(torch.float8_e4m3fn).view(torch.uint8)
        inside = (torch.arange(bs, device=dev)[None] < hn[:, None])[:, None, :, None]
        raw[hp] = torch.where(inside, again, raw[hp])
        raw[page, :, slot] = (x / fresh[page][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        scale[page] = fresh[page]
    return st["k"], st["v"], st["ks"], st["vs"]


def _attend(st):
    B, S, topk, H, G, hd, bs = (st[n] for n in ("B", "S", "topk", "H_kv", "G", "hd", "bs"))
    dev, rows = st["q"].device, B * S
    L = topk * bs
    q = st["q"].reshape(rows, H, G, hd)
    ids = st["ids"].reshape(rows, topk).long()
    seq = torch.arange(rows, device=dev) // S
    p = (st["q_start"][:, None] + torch.arange(S, device=dev)[None]).reshape(-1)
    hi = p if st["last"] is None else st["last"].reshape(-1)
    hi = torch.minimum(hi, st["ctx_len"][seq] - 1)
    lo = torch.zeros_like(p) if st["first"] is None else st["first"].reshape(-1)
    out = torch.empty_like(q)
    lse = torch.empty(rows, H, G, device=dev)
    mass = torch.empty(rows, H, topk, device=dev) if st["mass"] else None
    step = max(1, (1 << 28) // (L * H * hd))
    for r in range(0, rows, step):
        z = slice(r, r + step)
        n = ids[z].shape[0]
        page = st["table"][seq[z][:, None], ids[z].clamp(min=0)].long()
        pos = ids[z][:, :, None] * bs + torch.arange(bs, device=dev)
        keep = (ids[z][:, :, None] >= 0) & (pos >= lo[z][:, None, None]) & (pos <= hi[z][:, None, None])
        kk, vv = (torch.where(keep[:, :, None, :, None], pool.view(torch.uint8)[page].view(torch.float8_e4m3fn).float() * scale[page][:, :, :, None, None], 0.0)
                  .transpose(1, 2).reshape(n, H, L, hd) for pool, scale in ((st["k"], st["ks"]), (st["v"], st["vs"])))
        s = torch.matmul(q[z].float(), kk.transpose(2, 3)) * (1.0 / math.sqrt(hd))
        if st.get("cap"):
            s = st["cap"] * torch.tanh(s / st["cap"])
        if st["slopes"] is not None:
            s = s - st["slopes"].reshape(1, H, G, 1) * (p[z][:, None] - pos.reshape(n, L)).abs().float()[:, None, None, :]
        s = s.masked_fill(~keep.reshape(n, 1, 1, L), -math.inf)
        m = s.amax(dim=-1, keepdim=True)
        m = torch.where(m > -math.inf, m, torch.zeros_like(m))
        e = torch.exp(s - m)
        l = e.sum(dim=-1, keepdim=True)
        w = e / torch.where(l > 0, l, torch.ones_like(l))
        out[z] = torch.matmul(w, vv).to(out.dtype)
        lse[z] = (m * LOG2E + torch.log2(l)).squeeze(-1)
        if mass is not None:
            mass[z] = w.reshape(n, H, G, topk, bs).sum(dim=(2, 4))
    return (out.reshape(st["q"].shape), lse.reshape(B, S, H * G)) + ((mass.reshape(B, S, H, topk),) if mass is not None else ())


def _weigh(st):
    B, S, topk, NB = st["B"], st["S"], st["topk"], st["NB"]
    ids = st["ids"].reshape(B, S * topk).long()
    got = st["mass"].double().sum(dim=2).reshape(B, S * topk)
    got = torch.where(ids >= 0, got, torch.zeros_like(got))
    total = torch.zeros(B, NB, dtype=torch.float64, device=got.device).scatter_add_(1, ids.clamp(min=0), got)
    st["weight"].copy_((st["decay"] * st["weight"].double() + total).float())
    return (st["weight"],)


def _evict(st):
    B, NB, bs, budget, sink, recent = (st[n] for n in ("B", "NB", "bs", "budget", "sink", "recent"))
    weight, table, ctx = st["weight"], st["table"], st["ctx_len"]
    n = (ctx + bs - 1) // bs
    j = torch.arange(NB, device=ctx.device)[None]
    held = j < n[:, None]
    sure = held & ((j < sink) | (j >= n[:, None] - recent))
    rank = torch.where(sure, torch.full_like(weight, math.inf), weight)
    rank = torch.where(held, rank, torch.full_like(weight, -math.inf))
    order = torch.argsort(rank, dim=1, descending=True, stable=True)
    place = torch.empty_like(order).scatter_(1, order, j.expand(B, NB).contiguous())
    keep = held & (place < budget)
    # kept blocks first, then the freed ones, then what is not in use, each in order
    to = torch.argsort((~keep).long() + (~held).long(), dim=1, stable=True)
    kept = keep.sum(dim=1)
    freed = n - kept
    table_out = torch.gather(table, 1, to)
    weight_out = torch.where(j < kept[:, None], torch.gather(weight, 1, to), 0.0)
    kept_ids = torch.where(j < kept[:, None], to, -1)[:, :budget].to(torch.int32).contiguous()
    return table_out, (ctx - freed * bs).to(torch.int32), weight_out, kept_ids, freed.to(torch.int32)


def run(state):
    if own:
        return state["call"]()
    return {"append": _append, "attn": _attend, "scored": _attend, "weight": _weigh, "evict": _evict}[state["op"]](state)


# ---------------------------------------------------------------- 64 bits

def _dense(pool, scale, table_row, n, bs):
    """[H, n, hd]: one sequence's keys or values in 64 bits, in token order."""
    nb = -(-n // bs)
    pages = table_row[:nb].long()
    x = pool.view(torch.uint8)[pages].view(torch.float8_e4m3fn).to(torch.float64) * scale[pages].double()[:, :, None, None]
    return x.permute(1, 0, 2, 3).reshape(pool.shape[1], nb * bs, pool.shape[3])[:, :n]


def _exact_attn(c, st):
    H, G, hd, bs, S = c["H_kv"], c["G"], c["hd"], c["bs"], c["S"]
    if sum(_lens(c)) * S * H * G > 4e11 / 64:
        return None
    outs, lses, masses = [], [], []
    for b, n in enumerate(_lens(c)):
        K, V = (_dense(st[x], st[x + "s"], st["table"][b], n, bs) for x in "kv")
        nb = -(-n // bs)
        tok = torch.arange(n, device="cuda")
        step = max(1, int(1e8) // (G * n))
        for r in range(0, S, step):
            rows = torch.arange(r, min(S, r + step), device="cuda")
            m = len(rows)
            pick = torch.zeros(m, nb + 1, dtype=torch.bool, device="cuda")
            ids = st["ids"][b, rows].long()
            pick.scatter_(1, torch.where(ids >= 0, ids, nb), True)
            p = n - S + rows
            win = [_windows(c, int(x), n) for x in p.tolist()]
            lo, hi = (torch.tensor([w[i] for w in win], device="cuda") for i in (0, 1))
            see = pick[:, tok // bs] & (tok >= lo[:, None]) & (tok <= hi[:, None])
            for g in range(H):
                z = torch.einsum("mhd,td->mht", st["q"][b, rows, g * G:(g + 1) * G].double(), K[g]) / math.sqrt(hd)
                if c.get("cap"):
                    z = torch.tanh(z / c["cap"]) * c["cap"]
                if st["slopes"] is not None:
                    z = z - st["slopes"][g * G:(g + 1) * G].double()[None, :, None] * (p[:, None] - tok).abs().double()[:, None]
                z = torch.where(see[:, None], z, torch.tensor(-math.inf, dtype=torch.float64, device="cuda"))
                L = torch.logsumexp(z, dim=-1)
                w = torch.where(see[:, None], torch.exp(z - torch.where(L > -math.inf, L, 0.0)[..., None]), 0.0)
                outs.append(((b, r, g), torch.einsum("mht,td->mhd", w, V[g]).cpu()))
                lses.append(((b, r, g), (L * LOG2E).cpu()))
                if c["mass"]:
                    per = torch.zeros(m, nb * bs, dtype=torch.float64, device="cuda")
                    per[:, :n] = w.sum(dim=1)
                    per = per.reshape(m, nb, bs).sum(dim=2)
                    masses.append(((b, r, g), torch.where(ids >= 0, per.gather(1, ids.clamp(min=0)), 0.0).cpu()))
        del K, V
    B = c["B"]
    out, lse = torch.empty(B, S, H * G, hd, dtype=torch.float64), torch.empty(B, S, H * G, dtype=torch.float64)
    mass = torch.empty(B, S, H, c["topk"], dtype=torch.float64)
    for (b, r, g), x in outs:
        out[b, r:r + x.shape[0], g * G:(g + 1) * G] = x
    for (b, r, g), x in lses:
        lse[b, r:r + x.shape[0], g * G:(g + 1) * G] = x
    for (b, r, g), x in masses:
        mass[b, r:r + x.shape[0], g] = x
    return (out, lse) + ((mass,) if c["mass"] else ())


def _exact_append(c, st):
    """What each slot stands for before it is rounded, over the page's scale."""
    bs, counts, starts, got = c["bs"], _counts(c), _starts(c), {}
    for name in "kv":
        pool, scale, new = st[name].double(), st[name + "s"].double(), st[name + "_new"].double()
        for b in range(c["B"]):
            s, e = starts[b], starts[b] + counts[b]
            j0, j1 = s // bs, -(-e // bs)
            pages = st["table"][b, j0:j1].long()
            old = (pool[pages] * scale[pages][:, :, None, None]).permute(0, 2, 1, 3).reshape((j1 - j0) * bs, c["H_kv"], c["hd"])
            rows = torch.cat([old[: s - j0 * bs], new[b, : counts[b]]])
            fill = torch.zeros((j1 - j0) * bs - len(rows), c["H_kv"], c["hd"], dtype=torch.float64, device="cuda")
            fresh = torch.cat([torch.zeros_like(old[: s - j0 * bs]), new[b, : counts[b]], fill]).reshape(j1 - j0, bs, c["H_kv"], c["hd"])
            need = torch.exp2(torch.ceil(torch.log2(fresh.abs().amax(dim=(1, 3)).clamp(min=2.0 ** -70) / E4M3_MAX)).clamp(min=MIN_EXP))
            if s > j0 * bs:
                need[0] = torch.maximum(need[0], scale[pages[0]])
            full = torch.cat([rows, fill]).reshape(j1 - j0, bs, c["H_kv"], c["hd"]).permute(0, 2, 1, 3) / need[:, :, None, None]
            tail = torch.arange((j1 - j0) * bs, device="cuda").reshape(j1 - j0, 1, bs, 1) >= e - j0 * bs
            pool[pages] = torch.where(tail, pool[pages], full)
            scale[pages] = need
        got[name], got[name + "s"] = pool, scale
    return got["k"].cpu(), got["v"].cpu(), got["ks"].cpu(), got["vs"].cpu()


def exact(c, seed):
    st = prepare(c, seed)
    if c["op"] == "append":
        return _exact_append(c, st)
    if c["op"] in ("attn", "scored"):
        return _exact_attn(c, st)
    if c["op"] == "weight":
        total = st["weight"].double().cpu() * c["decay"]
        ids, mass = st["ids"].cpu().reshape(c["B"], -1), st["mass"].double().cpu().permute(0, 1, 3, 2).reshape(c["B"], -1, c["H_kv"])
        for b in range(c["B"]):
            on = ids[b] >= 0
            for g in range(c["H_kv"]):
                total[b] += torch.bincount(ids[b][on].long(), weights=mass[b, on, g], minlength=c["NB"])
        return (total,)
    left = []
    for b in range(c["B"]):
        w = st["weight"][b].tolist()
        n = -(-int(st["ctx_len"][b]) // c["bs"])
        keep = set(range(n))
        if n > c["budget"]:
            sure = set(range(min(c["sink"], n))) | set(range(max(0, n - c["recent"]), n))
            rest = sorted((j for j in range(n) if j not in sure), key=lambda j: (-w[j], j))
            keep = sure | set(rest[: c["budget"] - len(sure)])
        x = [w[j] for j in sorted(keep)]
        left.append(x + [0.0] * (c["NB"] - len(x)))
    return None, None, torch.tensor(left, dtype=torch.float64), None, None
