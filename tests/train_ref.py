"""Plain 64-bit implementations of the training pass (norm, rotation and cache write;
the attention's backward) and the error bounds that the kernels are held to (torch
float64, any device).

Norm and rotation.  r = 1/sqrt(mean(x^2) + eps) in fp32: D squares summed, at most
(D + 8) 2^-24 off, relatively; sine and cosine within 2^-21; three products and a sum:
  E = (D + 24) 2^-23 (|a| + |b|) |mscale|  for each rotated pair (a, b) of the normed
values, and the output's rounding to bf16 adds 2^-8 (|y| + E).
Backward: the rotated gradient is within 2^-20 (|da| + |db|) |mscale| =: 2^-20 A; with
sums of D products
  |dx - exact| <= (D + 32) 2^-22 r (|w| A + |x| r mean(|w| A |x| r)) + rounding,
  |dw - exact| <= (N + 64) 2^-23 sum A |x| r  over N rows.

Attention, backward.  Per (query i, token j), c_ij times listed:
  a score is D products summed in fp32 by tensor cores whose adders may truncate,
  |ds| <= (D + 8) 2^-23 S with S = max_j scale sum_d |q k|; lse is given in fp32 and
  enters in log2 units: P is within eps_p = 4 (D + 8) 2^-23 (S + |lse| + 4), relatively;
  P is rounded to bf16 for dV: (2^-8 + eps_p + (M + 16) 2^-23) sum_i P |dout|, M rows;
  dP is within (D + 8) 2^-23 sum |dout v|; delta, taken from the bf16 out, within
  2^-8 sum |dout out| + (D + 8) 2^-23 sum |dout out|;
  dS, rounded to bf16: E_ij = (2^-8 + eps_p) |dS| (1 + 2^-8) + P (1 + 2^-7) (dP's + delta's);
  dQ: scale (sum_j E |k| + (N + 16) 2^-23 sum |dS k|), dK alike over i; a query's parts
  of the selected blocks are rounded to bf16 before they are added (sparse): 2^-8 of
  each block's part;
and the outputs' rounding to bf16 adds 2^-8 (|x| + E).
"""
import math

import torch

BLOCK = 128
U = 2.0 ** -8


# ------------------------------------------------------ norm and rotation --
def angles(t, inv_freq):
    return t.double()[..., None] * torch.tensor(list(inv_freq), dtype=torch.float64, device=t.device)


def pair_dims(rot, interleaved, device):
    i = torch.arange(rot // 2, device=device)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(x, t, inv_freq, interleaved, mscale, sign=1.0):
    """x [B][T][heads][D] float64, positions t [B][T]."""
    rot = 2 * len(inv_freq)
    y = x.clone()
    if rot == 0:
        return y
    lo, hi = pair_dims(rot, interleaved, x.device)
    a = angles(t, inv_freq)[:, :, None]
    c, s = mscale * torch.cos(a), sign * mscale * torch.sin(a)
    y[..., lo] = x[..., lo] * c - x[..., hi] * s
    y[..., hi] = x[..., hi] * c + x[..., lo] * s
    return y


def pair_size(x, rot, interleaved, mscale):
    """|a| + |b| of each element's pair (its own size behind rot), times |mscale|."""
    y = x.abs()
    if rot:
        lo, hi = pair_dims(rot, interleaved, x.device)
        z = (y[..., lo] + y[..., hi]) * abs(mscale)
        y[..., lo], y[..., hi] = z, z
    return y


def norm_rope(x, w, t, inv_freq, interleaved, mscale, eps):
    """(values, bound) of the normed and rotated rows."""
    x = x.double()
    D = x.shape[-1]
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    y = rotate(x, t, inv_freq, interleaved, mscale)
    e = (D + 24) * 2.0 ** -23 * pair_size(x, 2 * len(inv_freq), interleaved, mscale)
    return y, e + U * (y.abs() + e)


def norm_rope_bwd(x, w, dy, t, inv_freq, interleaved, mscale, eps):
    """dx, its bound, dw, its bound (None without a norm)."""
    dy = dy.double()
    D, rot = dy.shape[-1], 2 * len(inv_freq)
    dn = rotate(dy, t, inv_freq, interleaved, mscale, -1.0)
    A = pair_size(dy, rot, interleaved, mscale)
    if w is None:
        e = 2.0 ** -20 * A
        return dn, e + U * (dn.abs() + e), None, None
    x, w = x.double(), w.double()
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    g = dn * w
    dx = r * (g - x * r * (g * x * r).mean(-1, keepdim=True))
    gA = w.abs() * A
    e = (D + 32) * 2.0 ** -22 * r * (gA + x.abs() * r * (gA * x.abs() * r).mean(-1, keepdim=True))
    n = dn.numel() // D
    dw = (dn * x * r).sum(dim=(0, 1, 2))
    ew = (n + 64) * 2.0 ** -23 * (A * x.abs() * r).sum(dim=(0, 1, 2))
    return dx, e + U * (dx.abs() + e), dw, ew


# ----------------------------------------------------------- attention -----
def counts_dense(T, N, q_start, device):
    t = q_start + torch.arange(T, device=device)
    return (torch.arange(N, device=device) <= t[:, None]).double()


def counts_sel(sel, N, q_start):
    """sel [T][16] of one (sequence, group): how often each query attends to each of
    N tokens (ids outside [0, lb] skipped)."""
    T, dev = sel.shape[0], sel.device
    t = q_start + torch.arange(T, device=dev)
    nb = -(-N // BLOCK)
    s = torch.where((sel >= 0) & (sel <= (t // BLOCK)[:, None]), sel, nb).long()
    c = torch.zeros(T, nb + 1, dtype=torch.float64, device=dev)
    c.scatter_add_(1, s, torch.ones_like(s, dtype=torch.float64))
    j = torch.arange(N, device=dev)
    return c[:, j // BLOCK] * (j <= t[:, None])


def forward(q, k, v, cnt, scale):
    """One head: out and lse (rows without a token: 0 and -inf)."""
    s = torch.where(cnt > 0, (q @ k.T) * scale + torch.log(cnt.clamp(min=1)), -torch.inf)
    lse = torch.logsumexp(s, -1)
    return torch.exp(s - torch.where(lse == -torch.inf, 0.0, lse)[:, None]) @ v, lse


def backward(q, k, v, out, dout, cnt, scale, sparse):
    """One head (all float64; out is the bf16 one): dq, dk, dv and their errors before
    the last rounding.  K and V rows that nobody attends to must be finite."""
    D, (R, N) = q.shape[-1], cnt.shape
    s = (q @ k.T) * scale
    exact, lse = forward(q, k, v, cnt, scale)
    p = torch.where(cnt > 0, cnt * torch.exp(s - torch.where(lse == -torch.inf, 0.0, lse)[:, None]), 0.0)
    dp = dout @ v.T
    ds = p * (dp - (dout * exact).sum(-1, keepdim=True))
    big = torch.where(cnt > 0, (q.abs() @ k.abs().T) * abs(scale), 0.0).amax(-1, keepdim=True)
    f = (D + 8) * 2.0 ** -23
    eps_p = 4 * f * (big + torch.where(lse == -torch.inf, 0.0, lse).abs()[:, None] + 4)
    e_dp = f * (dout.abs() @ v.abs().T)
    e_dl = (dout.abs() * (exact - out).abs()).sum(-1, keepdim=True) + f * (
        dout.abs() * exact.abs()).sum(-1, keepdim=True)
    e_ds = (U + eps_p) * ds.abs() * (1 + U) + p * (1 + 2 * U) * (e_dp + e_dl)
    seen_by = (cnt > 0).sum(0)[:, None]
    sees = (cnt > 0).sum(1)[:, None]
    a = abs(scale)
    e_dv = ((U + eps_p) * p).T @ dout.abs() + (seen_by + 16) * 2.0 ** -23 * (p.T @ dout.abs())
    e_dq = a * (e_ds @ k.abs() + (sees + 16) * 2.0 ** -23 * (ds.abs() @ k.abs()))
    e_dk = a * (e_ds.T @ q.abs() + (seen_by + 16) * 2.0 ** -23 * (ds.abs().T @ q.abs()))
    if sparse:
        for b in range(0, N, BLOCK):
            e_dq += U * a * (ds[:, b:b + BLOCK] @ k[b:b + BLOCK]).abs() * (1 + U)
    return (ds @ k * scale, ds.T @ q * scale, p.T @ dout), (e_dq, e_dk, e_dv)


def attn_backward(q, k, v, out, dout, q_start, kv_len, scale, sel=None):
    """q, out, dout [B][T][H][D], caches [B][blocks][128][G][D] (any float types).
    Returns dq, dk, dv (rows behind kv_len zero) and bounds, float64."""
    B, T, H, D = q.shape
    G = k.shape[3]
    dq = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    dk = torch.zeros(k.shape, dtype=torch.float64, device=q.device).flatten(1, 2)
    dv = torch.zeros_like(dk)
    eq, ek, ev = torch.zeros_like(dq), torch.zeros_like(dk), torch.zeros_like(dk)
    for b in range(B):
        N = q_start[b] + T
        for h in range(H):
            g = h // (H // G)
            cnt = counts_dense(T, N, q_start[b], q.device) if sel is None else \
                counts_sel(sel[b, :, g], N, q_start[b])
            r, e = backward(q[b, :, h].double(), k[b].flatten(0, 1)[:N, g].double(),
                            v[b].flatten(0, 1)[:N, g].double(), out[b, :, h].double(),
                            dout[b, :, h].double(), cnt, scale, sel is not None)
            dq[b, :, h], eq[b, :, h] = r[0], e[0]
            dk[b, :N, g] += r[1]
            ek[b, :N, g] += e[1]
            dv[b, :N, g] += r[2]
            ev[b, :N, g] += e[2]
    vals = dq, dk.view(k.shape), dv.view(k.shape)
    errs = eq, ek.view(k.shape), ev.view(k.shape)
    return vals, [e + U * (x.abs() + e) for x, e in zip(vals, errs)]


def attn_forward(q, k, v, q_start, scale, sel=None):
    """out (rounded to bf16) and lse (fp32) of every query, from 64-bit values."""
    B, T, H, D = q.shape
    G = k.shape[3]
    out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    for b in range(B):
        N = q_start[b] + T
        for h in range(H):
            g = h // (H // G)
            cnt = counts_dense(T, N, q_start[b], q.device) if sel is None else \
                counts_sel(sel[b, :, g], N, q_start[b])
            o, l = forward(q[b, :, h].double(), k[b].flatten(0, 1)[:N, g].double(),
                           v[b].flatten(0, 1)[:N, g].double(), cnt, scale)
            out[b, :, h], lse[b, :, h] = o.to(torch.bfloat16), l.float()
    return out, lse


def random_sel(T, G, q_start, gen, device, skew=0.3):
    """A selection as the index branch makes it, [B][T][G][16]: lb and the best 15
    blocks of a random score, ascending, -1 padded."""
    t = torch.tensor(q_start, device=device)[:, None] + torch.arange(T, device=device)
    nb = int(t.max()) // BLOCK + 1
    lb = (t // BLOCK)[:, :, None, None]
    kb = torch.arange(nb, device=device)
    score = torch.rand(*t.shape, G, nb, generator=gen, device=device)
    score = score + skew * torch.rand(t.shape[0], 1, G, nb, generator=gen, device=device)
    score = torch.where(kb < lb, score, torch.where(kb == lb, 9.0, -1.0))
    n = min(16, nb)
    top, ids = score.topk(n, dim=-1)
    ids = torch.where(top >= 0, ids, nb).sort(-1).values
    sel = torch.full((*t.shape, G, 16), -1, dtype=torch.int32, device=device)
    sel[..., :n] = torch.where(ids < nb, ids, -1).int()
    return sel


def check(got, want, bound, what=""):
    got = got.double()
    assert torch.isfinite(got).all(), what + ": non-finite outputs (unwritten rows?)"
    err = (got - want).abs()
    worst = (err / bound.clamp(min=1e-300)).max().item()
    assert (err <= bound).all(), "%s: error is %.3g of its bound" % (what, worst)
    return worst


def finite_difference(fn, x, dy, at, h=1e-4):
    """The derivative of sum(fn(x) dy) by central differences along the unit vector `at`."""
    up, down = fn(x + h * at), fn(x - h * at)
    return ((up - down) * dy).sum().item() / (2 * h)


def yarn_freqs(rot, base, factor, trained, fast=32.0, slow=1.0):
    """The by-parts frequencies, written from their definition: a pair that turns at
    least `fast` times within `trained` positions keeps its frequency, one below `slow`
    turns has it divided, linearly between in the pair's number."""
    def number(turns):
        # base^(-2 i / rot) trained / 2 pi = turns
        return rot / 2 * math.log(trained / (2 * math.pi * turns)) / math.log(base)
    lo, hi = max(math.floor(number(fast)), 0), min(math.ceil(number(slow)), rot - 1)
    out = []
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        keep = 1 - min(max((i - lo) / max(hi - lo, 1e-3), 0), 1)
        out.append(keep * f + (1 - keep) * f / factor)
    return out
