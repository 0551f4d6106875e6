"""Workloads of the training pass of an attention layer, and of the step that
writes its caches.

A case names its operator in "op":

append      msa_rope_append: the RMS norm of every query and key head, the rotary
            position, and the rows of K, V and K_idx written into the caches, in one
            pass over the projections
append_bwd  msa_rope_append_bwd: from the gradients of the rotated queries and of the
            caches to those of the projections and of the norms' weights
dense_bwd   msa_dense_attn_bwd: dQ, dK and dV of dense causal GQA attention
sparse_bwd  msa_sparse_attn_bwd: the same of the attention over the 16 selected blocks
            of every (query, group)

Positions and lengths are host integers, as the library takes them.  `own`
selects the framework's kernels; otherwise the operators run in their plain form
(elementary torch operations in 32 bits; the angles of far positions in 64).
"""
import math

import torch

own = False

BLOCK, TOPK = 128, 16
DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------ cases --
def _case(op, **kw):
    c = dict(op=op, B=1, T=1, H=48, G=8, D=128, Di=64, ctx=1, spread=0, rot=0, interleaved=False,
             base=10000.0, stretch=1.0, norm=True, fused=True, paged=False)
    c.update(kw)
    return c


def listed():
    return [
        # one decode step of 64 sequences of up to 4096 tokens: paged caches, the
        # projections as one tensor
        _case("append", name="append_step_64", B=64, T=1, ctx=4096, spread=4000, rot=128, paged=True),
        # a prefill chunk of 8192 tokens behind 777, half of each head rotated
        _case("append", name="append_chunk_8192", T=8192, ctx=8969, rot=64, paged=True),
        # ragged training sequences, interleaved pairs, positions stretched by 8, q, k and
        # v apart
        _case("append", name="append_1000_inter", B=3, T=1000, H=64, G=4, D=64, Di=32, ctx=6001,
              spread=5001, rot=64, interleaved=True, stretch=8.0, fused=False),
        # the backward pass of 8192 training tokens
        _case("append_bwd", name="append_bwd_8192", T=8192, ctx=8192, rot=128),
        # ... of two short sequences, 64 query / 4 KV heads of 64, a quarter rotated
        _case("append_bwd", name="append_bwd_301", B=2, T=301, H=64, G=4, D=64, Di=32, ctx=1201,
              spread=900, rot=16, fused=False),
        # dense layers: one training sequence of 16K tokens
        _case("dense_bwd", name="dense_bwd_16k", T=16384, ctx=16384),
        # four sequences of 2048 tokens
        _case("dense_bwd", name="dense_bwd_4x2048", B=4, T=2048, ctx=2048),
        # chunks of 1000 queries against ragged contexts, 64/4 heads of 64
        _case("dense_bwd", name="dense_bwd_chunk_1000", B=3, T=1000, H=64, G=4, D=64, Di=32, ctx=6001,
              spread=5001),
        # the smallest: one short sequence, one KV head
        _case("dense_bwd", name="dense_bwd_77", T=77, H=4, G=1, D=64, Di=32, ctx=77),
        # sparse layers: one training sequence of 8192 tokens
        _case("sparse_bwd", name="sparse_bwd_8192", T=8192, ctx=8192),
        # the last 2048 queries of a 32K context
        _case("sparse_bwd", name="sparse_bwd_chunk_2048", T=2048, ctx=32768),
        # a short chunk of two ragged sequences, 64/4 heads of 64
        _case("sparse_bwd", name="sparse_bwd_101", B=2, T=101, H=64, G=4, D=64, Di=32, ctx=5001,
              spread=2500),
    ]


_HEADS = [(48, 8), (64, 4), (4, 1), (12, 4), (8, 8), (16, 1), (10, 2)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "append_bwd", "dense_bwd", "dense_bwd", "sparse_bwd",
                     "sparse_bwd"])
    H, G = rng.choice(_HEADS)
    D, Di = rng.choice([64, 128]), rng.choice([32, 64])
    if rng.random() < 0.3:
        B, T = _log(rng, 1, 48), rng.randint(1, 8)
    else:
        B, T = rng.randint(1, 3), _log(rng, 5, 2500)
    ctx = T + (0 if rng.random() < 0.4 else _log(rng, 1, 9000 if B < 8 else 3000))
    if op in ("dense_bwd", "sparse_bwd"):
        ctx = max(ctx, 2)            # of one token alone every gradient but dv is zero
    kw = dict(B=B, T=T, H=H, G=G, D=D, Di=Di, ctx=ctx, spread=rng.randint(0, ctx - T))
    if op.startswith("append"):
        kw.update(rot=16 * rng.randint(0, D // 16), interleaved=rng.random() < 0.5,
                  base=rng.choice([10000.0, 1e6, 5e6]), stretch=rng.choice([1.0, 1.0, 4.0, 32.0]),
                  norm=rng.random() < 0.7, fused=rng.random() < 0.6)
        kw["paged"] = op == "append" and rng.random() < 0.5
    return _case(op, **kw)


# ------------------------------------------------------------ shared sizes --
def _lens(c):
    """Context length of each sequence: from ctx - spread to ctx, the first one ctx."""
    B, ctx, spread = c["B"], c["ctx"], c["spread"]
    return [ctx - (spread * i * 7919 // B) % (spread + 1) for i in range(B)]


def _max_blocks(c):
    return -(-c["ctx"] // BLOCK)


def work(case):
    c = case
    B, T, H, G, D, Di = (c[k] for k in ("B", "T", "H", "G", "D", "Di"))
    n = B * T
    if c["op"] == "append":
        return {"bytes": 2 * n * ((H + 2 * G) * D * 2 + Di * 2), "flops": 8 * n * (H + G) * D}
    if c["op"] == "append_bwd":
        # the inputs of the norm are read too, where there is one
        x = (H + G) * D * 2 if c["norm"] else 0
        return {"bytes": n * (x + 2 * (H + 2 * G) * D * 2), "flops": 16 * n * (H + G) * D}
    rows, pairs = 0, 0
    for m in _lens(c):
        rows += m
        for t in range(m - T, m):
            lb = t // BLOCK
            pairs += t + 1 if c["op"] == "dense_bwd" else min(lb, TOPK - 1) * BLOCK + t % BLOCK + 1
    # q, out, dout, dq and lse; k, v, dk and dv (five products of 2 D flops a pair)
    return {"bytes": n * H * (4 * 2 * D + 4) + 4 * rows * G * D * 2 +
            (4 * TOPK * n * G if c["op"] == "sparse_bwd" else 0), "flops": 10 * D * H * pairs}


# ----------------------------------------------------------------- inputs --
def _freqs(c):
    """Radians per position of each rotated pair."""
    return [c["base"] ** (-2.0 * i / c["rot"]) / c["stretch"] for i in range(c["rot"] // 2)]


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    B, T, H, G, D, Di = (c[k] for k in ("B", "T", "H", "G", "D", "Di"))
    mb = _max_blocks(c)
    lens = _lens(c)
    bf = dict(generator=g, device=DEV, dtype=torch.bfloat16)
    s = {"c": c, "lens": lens, "mb": mb, "handles": {}, "q_start": [n - T for n in lens]}
    s["q_start_dev"] = torch.tensor(s["q_start"], device=DEV)
    s["t"] = s["q_start_dev"][:, None] + torch.arange(T, device=DEV)          # [B][T]

    def projections(make):
        """q, k and v [B][T][heads][D]: parts of one tensor, or three."""
        if c["fused"]:
            return make(B, T, H + 2 * G, D).split([H, G, G], dim=2)
        return make(B, T, H, D), make(B, T, G, D), make(B, T, G, D)

    if c["op"].startswith("append"):
        size = 1 + 3 * torch.rand(B, T, 1, 1, generator=g, device=DEV)       # of a token's rows

        def values(*shape):
            return (torch.randn(*shape, **bf) * size).to(torch.bfloat16)

        s["q"], s["k"], s["v"] = projections(values)
        if c["norm"]:
            s["qw"] = (1 + 0.2 * torch.randn(D, generator=g, device=DEV)).to(torch.bfloat16)
            s["kw"] = (1 + 0.2 * torch.randn(D, generator=g, device=DEV)).to(torch.bfloat16)
        else:
            s["qw"] = s["kw"] = None
        pages = B * mb + (7 if c["paged"] else 0)
        s["pages"] = pages
        order = torch.randperm(pages, generator=g, device=DEV) if c["paged"] else \
            torch.arange(pages, device=DEV)
        s["table"] = order[:B * mb].reshape(B, mb).int()
        s["page"] = torch.gather(s["table"].long(), 1, s["t"] // BLOCK)       # [B][T]
        shape = (pages, BLOCK, G, D)
    if c["op"] == "append":
        s["ki"] = torch.randn(B, T, Di, **bf)
        s["k_cache"], s["v_cache"] = torch.randn(*shape, **bf), torch.randn(*shape, **bf)
        s["ki_cache"] = torch.randn(pages, BLOCK, Di, **bf)
        s["q_out"] = torch.empty(B, T, H, D, device=DEV, dtype=torch.bfloat16)
    elif c["op"] == "append_bwd":
        s["dq_out"] = torch.randn(B, T, H, D, **bf) * 0.01
        s["dk_cache"], s["dv_cache"] = torch.randn(*shape, **bf) * 0.1, torch.randn(*shape, **bf) * 0.1
        s["dq"], s["dk"], s["dv"] = projections(lambda *n: torch.empty(*n, device=DEV,
                                                                       dtype=torch.bfloat16))
        s["dqw"] = torch.empty(D, device=DEV) if c["norm"] else None
        s["dkw"] = torch.empty(D, device=DEV) if c["norm"] else None
    else:
        # scores of about two units, as of normed queries and keys
        s["q"] = torch.randn(B, T, H, D, **bf) * 2
        s["k"], s["v"] = (torch.randn(B, mb, BLOCK, G, D, **bf) for _ in range(2))
        s["dout"] = torch.randn(B, T, H, D, **bf) * 0.01
        s["dq"] = torch.empty(B, T, H, D, device=DEV, dtype=torch.bfloat16)
        s["dk"], s["dv"] = torch.zeros_like(s["k"]), torch.zeros_like(s["v"])
        s["sel"] = _selection(s, g) if c["op"] == "sparse_bwd" else None
        s["out"], s["lse"] = _forward(s)         # what the layer's forward pass left
    return s


def _selection(s, g):
    """lb and the 15 best of a score over the blocks before it: some blocks are
    chosen more than others, and the first one by nearly every query."""
    c, mb = s["c"], s["mb"]
    B, T, G = c["B"], c["T"], c["G"]
    lb = (s["t"] // BLOCK)[:, :, None, None]
    kb = torch.arange(mb, device=DEV)
    score = torch.rand(B, T, G, mb, generator=g, device=DEV)
    score += 0.3 * torch.rand(B, 1, G, mb, generator=g, device=DEV) + (kb == 0)
    score = torch.where(kb < lb, score, torch.where(kb == lb, 3.0, -1.0))
    n = min(TOPK, mb)
    top, ids = score.topk(n, dim=-1)
    ids = torch.where(top >= 0, ids, mb).sort(dim=-1).values
    sel = torch.full((B, T, G, TOPK), -1, dtype=torch.int32, device=DEV)
    sel[..., :n] = torch.where(ids < mb, ids, -1).int()
    return sel


# ------------------------------------------------------------ plain forms --
def _cos_sin(s):
    """[B][T][1][rot/2] each, the angles reduced in 64 bits."""
    f = torch.tensor(_freqs(s["c"]), device=DEV, dtype=torch.float64)
    a = s["t"].double()[..., None, None] * f
    return torch.cos(a).float(), torch.sin(a).float()


def _pairs(c, x):
    """The two halves of the rotated pairs of [..., D], and the dims behind them."""
    r = c["rot"]
    if c["interleaved"]:
        return x[..., 0:r:2], x[..., 1:r:2], x[..., r:]
    return x[..., :r // 2], x[..., r // 2:r], x[..., r:]


def _joined(c, a, b, rest):
    ab = torch.stack([a, b], -1).flatten(-2) if c["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([ab, rest], -1)


def _append(s):
    c = s["c"]
    cos, sin = _cos_sin(s)

    def rows(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
        a, b, rest = _pairs(c, x)
        return _joined(c, a * cos - b * sin, b * cos + a * sin, rest).to(torch.bfloat16)

    at = (s["page"], s["t"] % BLOCK)
    s["k_cache"][at] = rows(s["k"], s["kw"])
    s["v_cache"][at] = s["v"]
    s["ki_cache"][at] = s["ki"]
    return {"q": rows(s["q"], s["qw"]), "k": s["k_cache"], "v": s["v_cache"], "ki": s["ki_cache"]}


def _append_bwd(s):
    c = s["c"]
    cos, sin = _cos_sin(s)

    def rows(x, w, dy):
        a, b, rest = _pairs(c, dy.float())
        dn = _joined(c, a * cos + b * sin, b * cos - a * sin, rest)
        if w is None:
            return dn.to(torch.bfloat16), None
        x = x.float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        n = x * r
        dw = (dn * n).sum(dim=(0, 1, 2))
        dn = dn * w.float()
        return (r * (dn - n * (dn * n).mean(-1, keepdim=True))).to(torch.bfloat16), dw

    at = (s["page"], s["t"] % BLOCK)
    dq, dqw = rows(s["q"], s["qw"], s["dq_out"])
    dk, dkw = rows(s["k"], s["kw"], s["dk_cache"][at])
    return {"dq": dq, "dk": dk, "dv": s["dv_cache"][at], "dqw": dqw, "dkw": dkw}


def _tiles(s):
    """Runs of queries whose scores against all keys before them fit a few GB."""
    c = s["c"]
    step = max(1, min(c["T"], (1 << 30) // (c["B"] * c["H"] * s["mb"] * BLOCK)))
    top = max(s["q_start"])
    return [(i, min(i + step, c["T"]), top + min(i + step, c["T"])) for i in range(0, c["T"], step)]


def _seen(s, i0, i1, n):
    """Whether queries i0 .. i1 - 1 see keys 0 .. n - 1, [B][G or 1][1][queries][n]."""
    j = torch.arange(n, device=DEV)
    seen = (j <= s["t"][:, i0:i1, None])[:, None, None]
    if s["sel"] is None:
        return seen
    sel = s["sel"][:, i0:i1].long()
    chosen = torch.zeros(*sel.shape[:3], s["mb"] + 1, dtype=torch.bool, device=DEV)
    chosen.scatter_(-1, torch.where(sel < 0, s["mb"], sel), True)
    return seen & chosen.permute(0, 2, 1, 3)[:, :, None][..., j // BLOCK]


def _heads(c, x):
    """[B][T][H][D or nothing] -> [B][G][H/G][T][...] in 32 bits."""
    return x.float().unflatten(2, (c["G"], -1)).movedim(1, 3)


def _keys(x):
    """A cache [B][blocks][128][G][D] -> [B][G][1][rows][D] in 32 bits."""
    return x.flatten(1, 2).transpose(1, 2)[:, :, None].float()


def _forward(s):
    c = s["c"]
    q, k, v = _heads(c, s["q"]), _keys(s["k"]), _keys(s["v"])
    out, lse = torch.empty_like(q), torch.empty(q.shape[:-1], device=DEV)
    for i0, i1, n in _tiles(s):
        x = (q[..., i0:i1, :] @ k[..., :n, :].transpose(-1, -2)).mul_(c["D"] ** -0.5)
        x.masked_fill_(~_seen(s, i0, i1, n), -torch.inf)
        lse[..., i0:i1] = torch.logsumexp(x, -1)
        out[..., i0:i1, :] = x.sub_(lse[..., i0:i1, None]).exp_() @ v[..., :n, :]
    return (out.movedim(3, 1).flatten(2, 3).to(torch.bfloat16),
            lse.movedim(3, 1).flatten(2, 3).contiguous())


def _attn_bwd(s):
    c = s["c"]
    scale = c["D"] ** -0.5
    q, do, lse = _heads(c, s["q"]), _heads(c, s["dout"]), _heads(c, s["lse"])
    k, v = _keys(s["k"]), _keys(s["v"])
    dq, dk, dv = torch.empty_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for i0, i1, n in _tiles(s):
        qi, di, kn, vn = q[..., i0:i1, :], do[..., i0:i1, :], k[..., :n, :], v[..., :n, :]
        p = (qi @ kn.transpose(-1, -2)).mul_(scale).sub_(lse[..., i0:i1, None]).exp_()
        p.masked_fill_(~_seen(s, i0, i1, n), 0.0)
        # the heads of a group share K and V: their gradients add up
        dv[..., :n, :] += p.flatten(2, 3).transpose(-1, -2)[:, :, None] @ di.flatten(2, 3)[:, :, None]
        ds = di @ vn.transpose(-1, -2)
        # less their mean under p (out . dout, but for the rounding of out)
        ds.sub_((p * ds).sum(-1, keepdim=True)).mul_(p).mul_(scale)
        dk[..., :n, :] += ds.flatten(2, 3).transpose(-1, -2)[:, :, None] @ qi.flatten(2, 3)[:, :, None]
        dq[..., i0:i1, :] = ds @ kn

    def cache(x):
        return x[:, :, 0].transpose(1, 2).reshape(s["k"].shape).to(torch.bfloat16)

    return {"dq": dq.movedim(3, 1).flatten(2, 3).to(torch.bfloat16), "dk": cache(dk), "dv": cache(dv)}


# -------------------------------------------------- the framework's kernels --
def _handles(s):
    """Parameters, positions and workspace that a program keeps between calls."""
    h = s["handles"]
    if not h:
        import block_sparse_attention_04_gb300 as msa
        c = s["c"]
        h["msa"] = msa
        h["p"] = p = msa.params(c["B"], c["T"], c["H"], c["G"], c["D"], c["Di"], s["mb"])
        h["q_start"], h["kv_len"] = msa.positions(s["q_start"]), msa.positions(s["lens"])
        if c["op"].startswith("append"):
            h["rope"] = msa.rope(c["rot"], base=c["base"], interleaved=c["interleaved"],
                                 linear=c["stretch"], eps=EPS)
        h["ws"] = {"append": lambda: torch.empty(256, dtype=torch.uint8, device=DEV),
                   "append_bwd": lambda: msa.rope_append_bwd_workspace(p),
                   "dense_bwd": lambda: msa.dense_bwd_workspace(p),
                   "sparse_bwd": lambda: msa.sparse_bwd_workspace(p)}[c["op"]]()
    return h


def _own(s):
    c, h = s["c"], _handles(s)
    msa, p, ws = h["msa"], h["p"], h["ws"]
    if c["op"] == "append":
        paged = dict(block_table=s["table"], num_pool_blocks=s["pages"]) if c["paged"] else {}
        msa.msa_rope_append(p, h["rope"], s["q"], s["k"], s["v"], s["ki"], s["qw"], s["kw"],
                            h["q_start"], s["q_out"], s["k_cache"], s["v_cache"], s["ki_cache"], ws,
                            **paged)
        return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"], "ki": s["ki_cache"]}
    if c["op"] == "append_bwd":
        msa.msa_rope_append_bwd(p, h["rope"], s["q"], s["k"], s["qw"], s["kw"], h["q_start"],
                                s["dq_out"], s["dk_cache"], s["dv_cache"], s["dq"], s["dk"], s["dv"],
                                s["dqw"], s["dkw"], ws)
        return {k: s[k] for k in ("dq", "dk", "dv", "dqw", "dkw")}
    if c["op"] == "dense_bwd":
        msa.msa_dense_attn_bwd(p, s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], h["q_start"],
                               h["kv_len"], s["dq"], s["dk"], s["dv"], ws)
    else:
        msa.msa_sparse_attn_bwd(p, s["q"], s["k"], s["v"], s["sel"], s["out"], s["lse"], s["dout"],
                                h["q_start"], h["kv_len"], s["dq"], s["dk"], s["dv"], ws)
    return {k: s[k] for k in ("dq", "dk", "dv")}


_PLAIN = {"append": _append, "append_bwd": _append_bwd, "dense_bwd": _attn_bwd,
          "sparse_bwd": _attn_bwd}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["c"]["op"]](state)


# ------------------------------------------------------------ 64-bit values --
def _exact_rows(s, x, w):
    """The norm and the rotation of [B][T][heads][D] in 64 bits, by rotating each
    pair as a complex number."""
    c = s["c"]
    r = c["rot"]
    if w is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["D"] + EPS) * w
    if r == 0:
        return x
    f = torch.tensor([math.exp(-2.0 * i / r * math.log(c["base"])) / c["stretch"]
                      for i in range(r // 2)], device=DEV, dtype=torch.float64)
    turn = torch.polar(torch.ones((), device=DEV, dtype=torch.float64),
                       s["t"].double()[..., None, None] * f)
    i = torch.arange(r // 2, device=DEV)
    lo, hi = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + r // 2)
    z = torch.complex(x[..., lo], x[..., hi]) * turn
    y = x.clone()
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def _exact_append(s):
    out = {"q": _exact_rows(s, s["q"].double(), None if s["qw"] is None else s["qw"].double())}
    rows = {"k": _exact_rows(s, s["k"].double(), None if s["kw"] is None else s["kw"].double()),
            "v": s["v"].double(), "ki": s["ki"].double()}
    for name, x in rows.items():
        cache = s[name + "_cache"].double()
        for b, a in enumerate(s["q_start"]):
            t = a + torch.arange(s["c"]["T"], device=DEV)
            cache[s["table"][b].long()[t // BLOCK], t % BLOCK] = x[b]
        out[name] = cache
    return out


def _exact_append_bwd(s):
    c = s["c"]

    def grads(x, w, dy):
        x = x.double().requires_grad_()
        w = w if w is None else w.double().requires_grad_()
        with torch.enable_grad():
            y = _exact_rows(s, x, w)
        got = torch.autograd.grad(y, [x] if w is None else [x, w], dy.double())
        return got[0], None if w is None else got[1]

    def rows(cache):
        return torch.stack([cache[s["table"][b].long()].flatten(0, 1)[a:a + c["T"]]
                            for b, a in enumerate(s["q_start"])])

    dq, dqw = grads(s["q"], s["qw"], s["dq_out"])
    dk, dkw = grads(s["k"], s["kw"], rows(s["dk_cache"]))
    return {"dq": dq, "dk": dk, "dv": rows(s["dv_cache"]).double(), "dqw": dqw, "dkw": dkw}


def _exact_attn_bwd(s):
    """Gradients of softmax(q k / sqrt(D)) v by differentiating it, a group of heads and a
    run of queries at a time."""
    c = s["c"]
    T, H, G, D = (c[k] for k in ("T", "H", "G", "D"))
    dq = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    dk, dv = (torch.zeros(s["k"].shape, dtype=torch.float64, device=DEV).flatten(1, 2)
              for _ in range(2))
    hpg = H // G
    for b, a in enumerate(s["q_start"]):
        for g in range(G):
            hs = slice(g * hpg, (g + 1) * hpg)
            step = max(1, (1 << 25) // (hpg * s["lens"][b]))
            for i0 in range(0, T, step):
                i1 = min(T, i0 + step)
                n = a + i1
                t = torch.arange(a + i0, a + i1, device=DEV)
                j = torch.arange(n, device=DEV)
                seen = j <= t[:, None]
                if s["sel"] is not None:
                    mine = s["sel"][b, i0:i1, g]
                    seen = seen & (mine[:, :, None] == torch.arange(s["mb"], device=DEV)).any(1)[:, j // BLOCK]
                q = s["q"][b, i0:i1, hs].double().requires_grad_()
                k = s["k"][b].flatten(0, 1)[:n, g].double().requires_grad_()
                v = s["v"][b].flatten(0, 1)[:n, g].double().requires_grad_()
                with torch.enable_grad():
                    x = torch.einsum("ihd,jd->hij", q, k) / math.sqrt(D)
                    o = torch.einsum("hij,jd->ihd", torch.softmax(
                        torch.where(seen, x, -math.inf), -1), v)
                d = torch.autograd.grad(o, [q, k, v], s["dout"][b, i0:i1, hs].double())
                dq[b, i0:i1, hs] = d[0]
                dk[b, :n, g] += d[1]
                dv[b, :n, g] += d[2]
    return {"dq": dq, "dk": dk.view(s["k"].shape), "dv": dv.view(s["v"].shape)}


def exact(case, seed):
    c = case
    if c["op"].endswith("_bwd") and not c["op"].startswith("append"):
        # every key before a query is visited, chosen or not
        if 14 * c["D"] * c["H"] * c["T"] * sum(_lens(c)) > 4e12:
            return None
    s = prepare(case, seed)
    return {"append": _exact_append, "append_bwd": _exact_append_bwd, "dense_bwd": _exact_attn_bwd,
            "sparse_bwd": _exact_attn_bwd}[c["op"]](s)
