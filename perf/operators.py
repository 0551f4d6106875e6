"""Workloads of the serving operators around the block-major caches: the 8-bit
cache (its writer and the attention that reads it), attention over a sliding
window with a few first tokens that stay visible, and the page operations of a
paged pool.

A case names its operator in "op":

append   msa_cache_append_q8: new K and V rows, stored as e4m3 codes with one
         power-of-two scale per (128-token block, KV head)
sparse   msa_sparse_attn_q8: the 16 selected blocks of every (query, group),
         read from an 8-bit cache
window   msa_window_attn and msa_window_attn_q8: query t sees the tokens j <= t
         with j > t - window or j < sinks
fork     msa_pages_fork: rows of the block table that share another row's
         complete pages and get a copy of its last, partly filled one
compact  msa_pages_compact: live pages moved to the front of the pools

Caches are paged throughout: pools of 128-token pages and a block table.
Positions, lengths and row numbers are host integers, as the library takes
them.  `own` selects the framework's kernels; otherwise the operators run in
their plain form (elementary torch operations in 32 bits).
"""
import math

import torch

own = False

BLOCK, TOPK = 128, 16
MIN_EXP, MAX_EXP = -126, 119     # exponents of the 8-bit cache's scales
DEV = "cuda"


# ------------------------------------------------------------------ cases --
def _case(op, **kw):
    c = dict(op=op, B=1, T=1, H=48, G=8, D=128, Di=64, ctx=1, spread=0, window=0, sinks=0,
             q8=False, pages=0)
    c.update(kw)
    return c


def listed():
    return [
        # one decode step of 64 sequences of up to 4096 tokens: the step's new
        # token is appended; a quarter of them need a larger block scale
        _case("append", name="append_step_64", B=64, T=1, ctx=4096, spread=4000),
        # a prefill chunk appended behind 777 tokens: every block but the first whole
        _case("append", name="append_chunk_8192", B=1, T=8192, ctx=8969),
        # sparse attention of a decode step: 64 sequences of 32K tokens
        _case("sparse", name="sparse_step_64x32k", B=64, T=1, ctx=32768, spread=5000),
        # the smallest sparse call: one sequence, one token, 64 query / 4 KV heads
        _case("sparse", name="sparse_step_1", B=1, T=1, H=64, G=4, D=64, Di=32, ctx=5001),
        # sparse attention of a prefill chunk at the end of a 32K context
        _case("sparse", name="sparse_chunk_2048", B=1, T=2048, ctx=32768),
        # decode of 64 ragged sequences over a 4096-token window and 4 sinks, bf16 cache
        _case("window", name="window_step_64", B=64, T=1, ctx=16384, spread=14000, window=4096,
              sinks=4),
        # the smallest window call: one sequence, a 512-token window
        _case("window", name="window_step_1", B=1, T=1, H=4, G=1, D=64, Di=32, ctx=901,
              window=512),
        # the window reaches past every context (dense), 8-bit cache, 4 ragged sequences
        _case("window", name="full_step_4x64k_q8", B=4, T=1, ctx=65536, spread=40000,
              window=1 << 20, q8=True),
        # prefill of 16K tokens, window 4096 and 64 sinks, bf16 cache
        _case("window", name="window_prefill_16k", B=1, T=16384, ctx=16384, window=4096, sinks=64),
        # ragged chunks of 1000 queries on an 8-bit cache, odd window and sinks
        _case("window", name="window_chunk_1000_q8", B=3, T=1000, H=64, G=4, D=64, Di=32, ctx=6001,
              spread=5001, window=1000, sinks=5, q8=True),
        # 32 samples forked from prompts of up to 4000 tokens (bf16 pools)
        _case("fork", name="fork_32", B=32, ctx=4000, spread=3000, pages=2048),
        # an 8-bit pool of 4096 pages, 40 % of them live, compacted
        _case("compact", name="compact_4096", B=64, ctx=4096, spread=4000, pages=4096, q8=True),
    ]


_HEADS = [(48, 8), (64, 4), (4, 1), (12, 4), (8, 8), (16, 1), (10, 2)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "sparse", "sparse", "window", "window", "window", "fork",
                     "compact"])
    H, G = rng.choice(_HEADS)
    D, Di = rng.choice([64, 128]), rng.choice([32, 64])
    if op == "append":
        if rng.random() < 0.5:
            B, T = _log(rng, 1, 64), rng.randint(1, 4)
        else:
            B, T = rng.randint(1, 3), _log(rng, 5, 4000)
        ctx = T + _log(rng, 1, 4000)
        return _case(op, B=B, T=T, H=H, G=G, D=D, Di=Di, ctx=ctx, spread=rng.randint(0, ctx - T))
    if op == "sparse":
        if rng.random() < 0.6:
            B, T = _log(rng, 1, 64), rng.randint(1, 3)
            ctx = T + _log(rng, 1, 30000)
        else:
            B, T = rng.randint(1, 2), _log(rng, 20, 900)
            ctx = T + _log(rng, 1, 30000)
        return _case(op, B=B, T=T, H=H, G=G, D=D, Di=Di, ctx=ctx, spread=rng.randint(0, ctx - T))
    if op == "window":
        q8 = rng.random() < 0.5
        if rng.random() < 0.5:
            B, T = _log(rng, 1, 64), rng.randint(1, 4)
            ctx = T + _log(rng, 1, 16000)
        else:
            B, T = rng.randint(1, 2), _log(rng, 5, 4000)
            ctx = T + _log(rng, 1, 8000)
        w = rng.choice([_log(rng, 1, 6000), 1 << 20]) if ctx < 9000 else _log(rng, 1, 6000)
        return _case(op, B=B, T=T, H=H, G=G, D=D, Di=Di, ctx=ctx, spread=rng.randint(0, ctx - T),
                     window=w, sinks=rng.choice([0, 1, 4, rng.randint(1, 300)]), q8=q8)
    q8 = rng.random() < 0.5
    B = _log(rng, 1, 48)
    ctx = _log(rng, 1, 3500)
    need = B * (-(-ctx // BLOCK)) * 2 + B
    return _case(op, B=B, H=H, G=G, D=D, Di=Di, ctx=ctx, spread=rng.randint(0, ctx - 1), q8=q8,
                 pages=need + rng.randint(0, 300))


# ------------------------------------------------------------ shared sizes --
def _lens(c):
    """Context length of each sequence: from ctx - spread to ctx, the first one ctx."""
    B, ctx, spread = c["B"], c["ctx"], c["spread"]
    return [ctx - (spread * i * 7919 // B) % (spread + 1) for i in range(B)]


def _max_blocks(c):
    return -(-c["ctx"] // BLOCK)


def _visible(c, n):
    """Tokens that query t = n - 1 sees."""
    w = min(n, c["window"])
    return w + min(c["sinks"], n - w)


def work(case):
    c = case
    B, T, H, G, D, Di = (c[k] for k in ("B", "T", "H", "G", "D", "Di"))
    cb = 1 if c["q8"] or c["op"] == "sparse" else 2          # bytes of a cached value
    lens = _lens(c)
    if c["op"] == "append":
        n = B * T
        return {"bytes": n * (2 * G * D * (2 + 1) + 2 * Di * 2), "flops": 2 * n * G * D}
    if c["op"] == "sparse":
        flops, read = 0, 0
        for n in lens:
            for t in range(n - T, n):
                lb = t // BLOCK
                flops += 4 * D * H * (min(lb, TOPK - 1) * BLOCK + t % BLOCK + 1)
            # each query's own blocks for few queries, the whole context at most
            tok = min(-(-n // BLOCK), T * min(TOPK, (n - 1) // BLOCK + 1)) * BLOCK
            read += min(tok, n) * 2 * G * D
        return {"bytes": read + 2 * 2 * B * T * H * D + 4 * TOPK * B * T * G, "flops": flops}
    if c["op"] == "window":
        flops, read = 0, 0
        for n in lens:
            flops += sum(4 * D * H * _visible(c, t + 1) for t in range(n - T, n))
            first = max(0, n - T + 1 - c["window"])
            read += (n - first + min(c["sinks"], first)) * 2 * G * D * cb
        return {"bytes": read + 2 * 2 * B * T * H * D, "flops": flops}
    row = 2 * G * D * cb + 2 * Di                            # a token's bytes in all pools
    if c["op"] == "fork":
        part = sum(n % BLOCK for n in lens)
        return {"bytes": 2 * part * row + 8 * B * _max_blocks(c), "flops": 0}
    live = sum(-(-n // BLOCK) for n in lens)
    moved = live * (c["pages"] - live) // c["pages"]         # expected, pages placed at random
    return {"bytes": 2 * moved * BLOCK * row + 8 * (B * _max_blocks(c) + c["pages"]), "flops": 0}


# ----------------------------------------------------------------- inputs --
def _pools(c, g, pages, q8):
    G, D = c["G"], c["D"]

    def values(exp_lo, exp_hi):
        x = torch.randn(pages, BLOCK, G, D, generator=g, device=DEV, dtype=torch.bfloat16)
        if not q8:
            return x, None
        e = torch.randint(exp_lo, exp_hi, (pages, G), generator=g, device=DEV, dtype=torch.int8)
        return (x * 64).to(torch.float8_e4m3fn).view(torch.uint8), e

    k, ke = values(-8, -5)
    v, ve = values(-8, -4)
    ki = torch.randint(-8, 9, (pages, BLOCK, c["Di"]), generator=g, device=DEV).to(torch.bfloat16) / 8
    return {"k": k, "v": v, "ke": ke, "ve": ve, "ki": ki}


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    B, T, H, G, D, Di = (c[k] for k in ("B", "T", "H", "G", "D", "Di"))
    mb = _max_blocks(c)
    lens = _lens(c)
    s = {"c": c, "lens": lens, "mb": mb, "handles": {}}
    bf = dict(generator=g, device=DEV, dtype=torch.bfloat16)
    op = c["op"]
    if op in ("append", "sparse", "window"):
        pages = B * mb + 7
        s["pages"] = pages
        s["table"] = torch.randperm(pages, generator=g, device=DEV)[:B * mb].reshape(B, mb).int()
        s.update(_pools(c, g, pages, c["q8"] or op != "window"))
        s["q_start"] = [n - T for n in lens]
        s["q_start_dev"] = torch.tensor(s["q_start"], device=DEV)
    if op == "append":
        def rows():
            x = torch.randn(B, T, G, D, **bf)
            grow = torch.randint(0, 4, (B, 1, G, 1), generator=g, device=DEV) == 0
            return x * torch.where(grow, 16.0, 1.0).to(torch.bfloat16)
        s["k_new"], s["v_new"] = rows(), rows()
        s["ki_new"] = torch.randint(-8, 9, (B, T, Di), generator=g, device=DEV).to(torch.bfloat16) / 8
    elif op in ("sparse", "window"):
        s["q"] = torch.randn(B, T, H, D, **bf)
        s["out"] = torch.empty(B, T, H, D, device=DEV, dtype=torch.bfloat16)
    if op == "sparse":
        # lb and the best 15 of a random score over the blocks before it
        t = s["q_start_dev"][:, None] + torch.arange(T, device=DEV)
        lb = (t // BLOCK)[:, :, None, None]
        kb = torch.arange(mb, device=DEV)
        score = torch.rand(B, T, G, mb, generator=g, device=DEV)
        score = torch.where(kb < lb, score, torch.where(kb == lb, 2.0, -1.0))
        n = min(TOPK, mb)
        top, ids = score.topk(n, dim=-1)
        ids = torch.where(top >= 0, ids, mb).sort(dim=-1).values
        sel = torch.full((B, T, G, TOPK), -1, dtype=torch.int32, device=DEV)
        sel[..., :n] = torch.where(ids < mb, ids, -1).int()
        s["sel"] = sel
    if op in ("fork", "compact"):
        pages = c["pages"]
        s["pages"] = pages
        s.update(_pools(c, g, pages, c["q8"]))
        perm = torch.randperm(pages, generator=g, device=DEV).int()
        n = torch.tensor([-(-x // BLOCK) for x in lens], device=DEV)
        base = torch.cumsum(n, 0) - n
        kb = torch.arange(mb, device=DEV)
        used = kb < n[:, None]
        rows = torch.where(used, perm[(base[:, None] + kb).clamp(max=pages - 1)], -1).int()
        s["lens_dev"] = torch.tensor(lens, device=DEV)
        refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
        refs.scatter_add_(0, rows.clamp(min=0).long().reshape(-1), used.int().reshape(-1))
        if op == "fork":     # rows 0..B-1 hold the prompts, rows B..2B-1 receive the forks
            rows = torch.cat([rows, torch.full_like(rows, -1)])
            s["src"], s["dst"] = list(range(B)), list(range(B, 2 * B))
            s["src_dev"] = torch.arange(B, device=DEV)
            s["dst_dev"] = torch.arange(B, 2 * B, device=DEV)
        else:
            s["table_out"] = torch.empty_like(rows)
            s["refs_out"] = torch.empty_like(refs)
            s["live"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        s["table"], s["refs"] = rows.contiguous(), refs
    return s


# ------------------------------------------------------------ plain forms --
def _pow2(e):
    return torch.ldexp(torch.ones((), device=DEV), e.float())


def _value(x, e, page, *where):
    """Cached values at [page, *where, :, :] as fp32: x [pages][128][G][D]."""
    v = x[(page, *where)]
    if e is None:
        return v.float()
    return v.view(torch.float8_e4m3fn).float() * _pow2(e[page])[..., None]


def _append(s):
    c = s["c"]
    B, T, G, D = c["B"], c["T"], c["G"], c["D"]
    nb = (T + 2 * BLOCK - 2) // BLOCK            # blocks that T rows can touch
    first = s["q_start_dev"] // BLOCK
    kb = first[:, None] + torch.arange(nb, device=DEV)
    t = (kb[..., None] * BLOCK + torch.arange(BLOCK, device=DEV))          # [B][nb][128]
    i = t - s["q_start_dev"][:, None, None]
    new = (i >= 0) & (i < T)
    old = i < 0
    b = torch.arange(B, device=DEV)[:, None]
    page = s["table"][b, kb.clamp(max=s["mb"] - 1)].long()
    touched = new.any(-1)
    bi = b[..., None].expand_as(i), i.clamp(0, T - 1)
    for x, codes, exps in ((s["k_new"], s["k"], s["ke"]), (s["v_new"], s["v"], s["ve"])):
        x = x[bi].float()                                                # [B][nb][128][G][D]
        fresh = new[..., None, None]
        amax = torch.where(fresh & x.isfinite(), x.abs(), 0.0).amax(dim=(2, 4))  # [B][nb][G]
        m, e = torch.frexp(amax)
        need = torch.where(amax > 0, torch.where(m <= 0.875, e - 9, e - 8), MIN_EXP)
        need = need.clamp(MIN_EXP, MAX_EXP)
        had = old.any(-1)[..., None]
        before = exps[page].int()
        after = torch.where(had, torch.maximum(need, before), need)
        kept = codes[page].view(torch.float8_e4m3fn).float() * _pow2(before - after)[:, :, None, :, None]
        fits = 448.0 * _pow2(after)[:, :, None, :, None]
        x = torch.where(x.isfinite(), torch.minimum(torch.maximum(x, -fits), fits), torch.nan)
        rows = torch.where(fresh, x * _pow2(-after)[:, :, None, :, None], kept)
        rows = rows.to(torch.float8_e4m3fn).view(torch.uint8)
        grown = had & (after > before)           # only then do the earlier rows change
        keep = ~(fresh | (old[..., None, None] & grown[:, :, None, :, None]))
        rows = torch.where(keep, codes[page], rows)
        codes[page[touched]] = rows[touched]
        exps[page[touched]] = after[touched].to(torch.int8)
    s["ki"][page[..., None].expand_as(t)[new], (t % BLOCK)[new]] = s["ki_new"][bi][new]
    return _cache_state(s)


def _cache_state(s):
    return {"k": s["k"].view(torch.float8_e4m3fn), "v": s["v"].view(torch.float8_e4m3fn),
            "ke": s["ke"], "ve": s["ve"], "ki": s["ki"]}


def _attend(q, k, v, seen, scale):
    """q [..., G, R, D] of R (query, head) rows, k and v [..., G, N, D], seen [..., G or 1, R, N];
    a row that sees nothing is 0."""
    x = (q @ k.transpose(-1, -2)).mul_(scale)
    x.masked_fill_(~seen, -torch.inf)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(m.masked_fill(m == -torch.inf, 0.0)).exp_()
    l = x.sum(-1, keepdim=True)
    return (x @ v) / torch.where(l == 0, 1.0, l)


def _sparse(s):
    c = s["c"]
    B, T, H, G, D = (c[k] for k in ("B", "T", "H", "G", "D"))
    t = s["q_start_dev"][:, None] + torch.arange(T, device=DEV)
    sel = s["sel"].long()                                       # [B][T][G][16]
    b = torch.arange(B, device=DEV)[:, None, None, None]
    page = s["table"][b, sel.clamp(min=0)].long()
    g = torch.arange(G, device=DEV)[:, None]

    def gathered(codes, exps):                                  # [B][T][G][16*128][D]
        x = codes.transpose(1, 2)[page, g].view(torch.float8_e4m3fn).float()
        return x.mul_(_pow2(exps[page, g])[..., None, None]).flatten(3, 4)

    tok = sel[..., None] * BLOCK + torch.arange(BLOCK, device=DEV)
    seen = ((sel[..., None] >= 0) & (tok <= t[:, :, None, None, None])).flatten(3)
    q = s["q"].float().view(B, T, G, H // G, D)
    o = _attend(q, gathered(s["k"], s["ke"]), gathered(s["v"], s["ve"]), seen[..., None, :],
                D ** -0.5)
    return o.reshape(B, T, H, D).to(torch.bfloat16)


def _window(s):
    c = s["c"]
    B, T, H, G, D, W = (c[k] for k in ("B", "T", "H", "G", "D", "window"))
    top = max(s["lens"])
    W = min(W, top)
    tile = min(T, 512)                           # queries that share a span of keys
    nt = -(-T // tile)
    i = torch.arange(nt * tile, device=DEV).view(nt, tile)
    t = s["q_start_dev"][:, None, None] + i                      # [B][nt][tile]
    span = t[..., :1] - (W - 1) + torch.arange(tile + W - 1, device=DEV)
    sinks = torch.arange(min(c["sinks"], top), device=DEV).expand(B, nt, -1)
    j = torch.cat([sinks, span], -1)                             # [B][nt][N]
    ok = (j >= 0) & (j <= (s["q_start_dev"] + T - 1)[:, None, None])
    jc = torch.where(ok, j, 0)
    b = torch.arange(B, device=DEV)[:, None, None]
    page = s["table"][b, jc // BLOCK].long()
    kv = [_value(x, e, page, jc % BLOCK).transpose(2, 3)         # [B][nt][G][N][D]
          for x, e in ((s["k"], s["ke"]), (s["v"], s["ve"]))]
    lo = t - W + 1
    jn, tn, ln = j[:, :, None, :], t[..., None], lo[..., None]
    is_sink = torch.arange(j.shape[-1], device=DEV) < sinks.shape[-1]
    seen = ok[:, :, None, :] & (jn <= tn) & torch.where(is_sink, jn < ln, jn >= ln)
    q = s["q"].float()
    if nt * tile > T:
        q = torch.cat([q, q.new_zeros(B, nt * tile - T, H, D)], 1)
    q = q.view(B, nt, tile, G, H // G, D).permute(0, 1, 3, 4, 2, 5).reshape(B, nt, G, -1, D)
    seen = seen[:, :, None, None].expand(-1, -1, 1, H // G, -1, -1).flatten(3, 4)
    o = _attend(q, kv[0], kv[1], seen, D ** -0.5)
    o = o.view(B, nt, G, H // G, tile, D).permute(0, 1, 4, 2, 3, 5).reshape(B, nt * tile, H, D)
    return o[:, :T].to(torch.bfloat16)


def _pool_list(s):
    return [s[k] for k in ("k", "v", "ki", "ke", "ve") if s[k] is not None]


def _page_state(s, table, refs, **more):
    r = {k: s[k] for k in ("ki", "ke", "ve") if s[k] is not None}
    for k in ("k", "v"):
        r[k] = s[k] if s["ke"] is None else s[k].view(torch.float8_e4m3fn)
    return {**r, "table": table, "refs": refs, **more}


def _fork(s):
    table, refs, pages = s["table"], s["refs"], s["pages"]

    def count(ids, by):
        ok = (ids >= 0) & (ids < pages)
        refs.scatter_add_(0, torch.where(ok, ids, 0).long().reshape(-1),
                          torch.where(ok, by, 0).int().reshape(-1))

    count(table[s["dst_dev"]], torch.full((), -1, device=DEV))
    n = s["lens_dev"]
    kb = torch.arange(s["mb"], device=DEV)
    src = table[s["src_dev"]]
    whole = kb < (n // BLOCK)[:, None]
    rows = torch.where(whole, src, -1)
    count(rows, torch.ones((), device=DEV, dtype=torch.int32))
    part = [j for j, x in enumerate(s["lens"]) if x % BLOCK]
    if part:
        pj = torch.tensor(part, device=DEV)
        ids = torch.arange(pages, device=DEV)
        free = torch.where(refs == 0, ids, pages).topk(len(part), largest=False, sorted=True).values
        old = src[pj, n[pj] // BLOCK].long()
        rows[pj, n[pj] // BLOCK] = free.int()
        refs[free] = 1
        row = torch.arange(BLOCK, device=DEV) < (n[pj] % BLOCK)[:, None]
        for x in _pool_list(s):
            if x.dim() > 2:
                mask = row.view(*row.shape, *[1] * (x.dim() - 2))
                x[free] = torch.where(mask, x[old], x[free])
            else:
                x[free] = x[old]
    table[s["dst_dev"]] = rows
    return _page_state(s, table, refs)


def _compact(s):
    refs, table, pages = s["refs"], s["table"], s["pages"]
    ids = torch.arange(pages, device=DEV)
    live = refs > 0
    n = live.sum()
    src = (live & (ids >= n)).nonzero()[:, 0]
    dst = (~live & (ids < n)).nonzero()[:, 0]
    to = ids.clone()
    to[src] = dst
    for x in _pool_list(s):
        x[dst] = x[src]
    ok = (table >= 0) & (table < pages)
    out = torch.where(ok, to[torch.where(ok, table, 0).long()].int(), table)
    refs_out = torch.zeros_like(refs)
    refs_out[to[live]] = refs[live]              # live pages only: their places are distinct
    return _page_state(s, out, refs_out, live=n.int().reshape(1))


# -------------------------------------------------- the framework's kernels --
def _handles(s, make):
    """Parameters, positions and workspace that a program keeps between calls."""
    h = s["handles"]
    if not h:
        import block_sparse_attention_04_gb300 as msa
        c = s["c"]
        h["msa"] = msa
        h["p"] = msa.params(c["B"], c["T"], c["H"], c["G"], c["D"], c["Di"], s["mb"])
        make(h, msa)
    return h


def _own(s):
    c = s["c"]
    op = c["op"]
    paged = dict(block_table=s["table"], num_pool_blocks=s["pages"])

    def make(h, msa):
        if op in ("append", "sparse", "window"):
            h["q_start"], h["kv_len"] = msa.positions(s["q_start"]), msa.positions(s["lens"])
        if op == "append":
            h["ws"] = torch.empty(256, dtype=torch.uint8, device=DEV)
        elif op == "sparse":
            h["ws"] = msa.q8_workspace(h["p"])
        elif op == "window":
            h["ws"] = msa.window_workspace(h["p"])
        else:
            h["ws"] = msa.pages_workspace(s["pages"])
            h["pools"] = msa.pools(_pool_list(s))

    h = _handles(s, make)
    msa, p, ws = h["msa"], h["p"], h["ws"]
    if op == "append":
        msa.msa_cache_append_q8(p, s["k_new"], s["v_new"], s["ki_new"], h["q_start"], s["k"], s["v"],
                                s["ke"], s["ve"], s["ki"], ws, **paged)
        return _cache_state(s)
    if op == "sparse":
        msa.msa_sparse_attn_q8(p, s["q"], s["k"], s["v"], s["ke"], s["ve"], s["sel"], h["q_start"],
                               h["kv_len"], s["out"], ws, **paged)
        return s["out"]
    if op == "window" and c["q8"]:
        msa.msa_window_attn_q8(p, c["window"], c["sinks"], s["q"], s["k"], s["v"], s["ke"], s["ve"],
                               h["q_start"], h["kv_len"], s["out"], ws, **paged)
        return s["out"]
    if op == "window":
        msa.msa_window_attn(p, c["window"], c["sinks"], s["q"], s["k"], s["v"], h["q_start"],
                            h["kv_len"], s["out"], ws, **paged)
        return s["out"]
    if op == "fork":
        msa.msa_pages_fork(h["pools"], s["pages"], s["table"], s["refs"], s["src"], s["dst"],
                           s["lens"], ws)
        return _page_state(s, s["table"], s["refs"])
    msa.msa_pages_compact(h["pools"], s["pages"], s["table"], s["refs"], s["table_out"],
                          s["refs_out"], s["live"], ws)
    return _page_state(s, s["table_out"], s["refs_out"], live=s["live"])


_PLAIN = {"append": _append, "sparse": _sparse, "window": _window, "fork": _fork,
          "compact": _compact}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["c"]["op"]](state)


# ------------------------------------------------------------ 64-bit values --
def _exact_append(s):
    c = s["c"]
    T = c["T"]
    f8 = torch.float8_e4m3fn
    out = {k: s[k].clone() for k in ("ke", "ve", "ki")}
    for x, name, en in ((s["k_new"], "k", "ke"), (s["v_new"], "v", "ve")):
        vals = s[name].view(f8).double()
        for b, a in enumerate(s["q_start"]):
            for kb in range(a // BLOCK, (a + T - 1) // BLOCK + 1):
                page = int(s["table"][b, kb])
                r0, r1 = max(a - kb * BLOCK, 0), min(a + T - kb * BLOCK, BLOCK)
                rows = x[b, kb * BLOCK + r0 - a:kb * BLOCK + r1 - a].double()      # [r][G][D]
                amax = rows.abs().amax(dim=(0, 2))
                e = torch.ceil(torch.log2(torch.clamp(amax, min=1e-300) / 448))
                e = torch.where(amax > 448 * 2.0 ** e, e + 1, e)
                e = torch.where(amax <= 448 * 2.0 ** (e - 1), e - 1, e).clamp(MIN_EXP, MAX_EXP)
                if r0 > 0:
                    before = out[en][page].double()
                    e = torch.maximum(e, before)
                    grown = (e > before)[None, :, None]
                    was = vals[page, :r0]
                    now = (was * 2.0 ** (before - e)[None, :, None]).float().to(f8).double()
                    vals[page, :r0] = torch.where(grown, now, was)
                vals[page, r0:r1] = (rows * 2.0 ** (-e)[None, :, None]).float().to(f8).double()
                out[en][page] = e.to(torch.int8)
        out[name] = vals
    for b, a in enumerate(s["q_start"]):
        for kb in range(a // BLOCK, (a + T - 1) // BLOCK + 1):
            r0, r1 = max(a - kb * BLOCK, 0), min(a + T - kb * BLOCK, BLOCK)
            i = kb * BLOCK - a
            out["ki"][int(s["table"][b, kb]), r0:r1] = s["ki_new"][b, i + r0:i + r1]
    return {**out, "ke": None, "ve": None, "ki": out["ki"].double()}


def _cache64(s, b, g):
    """Sequence b's K and V of KV head g, every row of its pages, in 64 bits."""
    page = s["table"][b].long()
    r = []
    for x, e in ((s["k"], s["ke"]), (s["v"], s["ve"])):
        if e is None:
            r.append(x[page, :, g].double().flatten(0, 1))
        else:
            y = x[page, :, g].view(torch.float8_e4m3fn).double()
            r.append((y * (2.0 ** e[page, g].double())[:, None, None]).flatten(0, 1))
    return r


def _exact_attention(s, seen_of, tile):
    c = s["c"]
    B, T, H, G, D = (c[k] for k in ("B", "T", "H", "G", "D"))
    hpg = H // G
    out = torch.empty(B, T, H, D, dtype=torch.float64, device=DEV)
    for b in range(B):
        for g in range(G):
            k, v = _cache64(s, b, g)
            for i0 in range(0, T, tile):
                i1 = min(T, i0 + tile)
                a, z, seen = seen_of(b, g, i0, i1)               # keys [a, z), [queries][z - a]
                q = s["q"][b, i0:i1, g * hpg:(g + 1) * hpg].double()
                x = torch.einsum("ihd,jd->ihj", q, k[a:z]) / math.sqrt(D)
                x = torch.where(seen[:, None, :], x, -math.inf)
                w = torch.softmax(x, dim=-1)
                out[b, i0:i1, g * hpg:(g + 1) * hpg] = torch.einsum("ihj,jd->ihd", w, v[a:z])
    return out


def _exact_sparse(s):
    n = s["mb"] * BLOCK
    j = torch.arange(n, device=DEV)

    def seen_of(b, g, i0, i1):
        t = s["q_start"][b] + torch.arange(i0, i1, device=DEV)
        chosen = (s["sel"][b, i0:i1, g, :, None] == torch.arange(s["mb"], device=DEV)).any(1)
        return 0, n, chosen[:, j // BLOCK] & (j <= t[:, None])

    return _exact_attention(s, seen_of, 256)


def _exact_window(s):
    c = s["c"]
    W, S, T = c["window"], c["sinks"], c["T"]

    def seen_of(b, g, i0, i1):
        t = s["q_start"][b] + torch.arange(i0, i1, device=DEV)
        z = s["q_start"][b] + i1
        a = 0 if S else max(0, s["q_start"][b] + i0 - W + 1)
        j = torch.arange(a, z, device=DEV)
        return a, z, (j <= t[:, None]) & ((j > t[:, None] - W) | (j < S))

    return _exact_attention(s, seen_of, 1024)


def exact(case, seed):
    op = case["op"]
    if op in ("fork", "compact"):
        return None              # pages are moved as they are, nothing is computed
    flops = work(case)["flops"]
    if op == "window":           # every key up to the tile's end is visited when sinks stay visible
        flops = sum(4 * case["D"] * case["H"] * case["T"] * n for n in _lens(case))
    if op == "sparse":
        flops = 4 * case["D"] * case["H"] * case["B"] * case["T"] * case["ctx"]
    if flops > 1.2e13 or (op == "append" and case["B"] * (case["T"] // BLOCK + 1) > 2000):
        return None
    s = prepare(case, seed)
    return {"append": _exact_append, "sparse": _exact_sparse, "window": _exact_window}[op](s)
