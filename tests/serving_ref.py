"""Plain 64-bit implementations of the serving operators, and the error bounds
that the kernels are held to (torch float64, any device).

Attention bound.  Write w_j for the exact softmax weights of a row and
A = sum_j w_j |v_j| (per output element).  A kernel rounds
  - each weight p to bf16 before the product with V: u_p = 2^-8, relative,
    contributing u_p A;
  - each score: D products summed in fp32 by the tensor cores, whose adders may
    truncate (2^-23 per term), and an 8-bit call's Q to f16 after scaling the
    row's maximum to 2^13 (elements below 2^-14 round at 2^-25 absolute, i.e.
    2^-38 of the maximum, below a term's 2^-23): |ds| <= (D + 8) 2^-23 S with
    S = max_j scale sum_d |q_d k_jd|; a weight moves by at most 2 |ds|
    relatively (once in p, once in the normaliser), doubled for second order;
  - exponentials (2^-22 relative) and sums over N tokens in fp32:
    (N + 16) 2^-23.
  E = (u_p + 4 (D + 8) 2^-23 S + (N + 16) 2^-23) A, and the output's rounding to
bf16 adds 2^-8 (|o| + E):  |got - o| <= E + 2^-8 (|o| + E).
"""
import numpy as np
import torch

BLOCK = 128
MIN_EXP, MAX_EXP = -126, 119
U_BF16 = 2.0 ** -8


def codes_to_f64(codes):
    return codes.view(torch.float8_e4m3fn).to(torch.float32).double()


def dequant(codes, exps):
    """codes uint8 [..., 128, G, D], exps int8 [..., G] -> float64."""
    e = exps.double().clamp(MIN_EXP, MAX_EXP)
    return codes_to_f64(codes) * torch.pow(2.0, e)[..., None, :, None]


def attention(q, k, v, seen, scale, u_p):
    """One sequence's rows.  q [R][D], k and v [N][D], seen [R][N] (float64,
    bool).  Returns (o, bound), rows that see nothing as zeros (bound 0).
    Values of tokens that a row does not see are never used."""
    D = q.shape[-1]
    any_seen = seen.any(0)
    k = torch.where(any_seen[:, None], k, 0.0)
    v = torch.where(any_seen[:, None], v, 0.0)
    s = (q @ k.T) * scale
    s = torch.where(seen, s, -torch.inf)
    empty = ~seen.any(-1, keepdim=True)
    w = torch.softmax(torch.where(empty, 0.0, s), -1)
    w = torch.where(seen, w, 0.0)
    o = w @ v
    a = w @ v.abs()
    big = torch.where(seen, (q.abs() @ k.abs().T) * abs(scale), 0.0).amax(-1, keepdim=True)
    n = seen.sum(-1, keepdim=True).double()
    e = (u_p + 4 * (D + 8) * 2.0 ** -23 * big + (n + 16) * 2.0 ** -23) * a
    return o, e + 2.0 ** -8 * (o.abs() + e)


def rows_of(pool, table, b):
    """Sequence b's cache rows [max_blocks*128][G][D] through a table (or None)."""
    nb = pool.shape[1] if table is None else None
    x = pool[b] if nb is not None else pool[table[b].long()]
    return x.reshape(-1, *x.shape[-2:])


def attend_call(q, k, v, q_start, seen_of, scale, u_p):
    """q [B][T][H][D]; k, v: per sequence float64 [N][G][D]; seen_of(b, g, t)
    -> [T][N] for positions t [T].  Returns (o, bound) [B][T][H][D]."""
    B, T, H, D = q.shape
    G = k[0].shape[1]
    o = torch.empty(q.shape, dtype=torch.float64, device=q.device)
    bound = torch.empty_like(o)
    for b in range(B):
        t = q_start[b] + torch.arange(T, device=q.device)
        for h in range(H):
            g = h // (H // G)
            o[b, :, h], bound[b, :, h] = attention(q[b, :, h].double(), k[b][:, g], v[b][:, g],
                                                   seen_of(b, g, t), scale, u_p)
    return o, bound


def window_seen(N, window, sinks, device):
    j = torch.arange(N, device=device)

    def seen(b, g, t):
        t = t[:, None]
        return (j <= t) & ((j > t - window) | (j < sinks))
    return seen


def sel_seen(sel, N, device):
    j = torch.arange(N, device=device)
    blocks = torch.arange(-(-N // BLOCK), device=device)

    def seen(b, g, t):
        chosen = (sel[b, :, g, :, None] == blocks).any(1)
        return chosen[:, j // BLOCK] & (j <= t[:, None])
    return seen


def check(got, want, bound):
    got = got.double()
    assert torch.isfinite(got).all(), "non-finite outputs (unwritten rows?)"
    err = (got - want).abs()
    worst = (err / bound.clamp(min=1e-300)).max().item()
    assert (err <= bound).all(), "error is %.3g of its bound" % worst
    return worst


# ---------------------------------------------------------- 8-bit writer --
def need_exp(amax):
    """The smallest e in [MIN_EXP, MAX_EXP] with amax <= 448 * 2^e, by search."""
    for e in range(MIN_EXP, MAX_EXP + 1):
        if amax <= 448.0 * 2.0 ** e:
            return e
    return MAX_EXP


def round_e4m3(x):
    """float64 array -> e4m3 codes (uint8), round to nearest even, saturating at
    448; NaN and infinities as 0x7F.  By search over the 127 finite codes."""
    mag = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10)
                    for c in range(0x7F)])
    x = np.asarray(x, np.float64)
    bad = ~np.isfinite(x)
    a = np.minimum(np.abs(np.where(bad, 0, x)), 448.0)
    hi = np.searchsorted(mag, a, side="left").clip(0, 0x7E)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - mag[lo], mag[hi] - a
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = pick.astype(np.uint8) | np.where(np.signbit(x) & ~bad, 0x80, 0).astype(np.uint8)
    return np.where(bad, np.uint8(0x7F), code).astype(np.uint8)


def decode_e4m3(c):
    c = np.asarray(c)
    m = (c & 0x7F).astype(np.int64)
    v = np.where(m < 8, m * 2.0 ** -9, (8 + (m & 7)) * np.exp2((m >> 3) - 10.0))
    v = np.where(m == 0x7F, np.nan, v)
    return np.where(c & 0x80, -v, v)


def append(codes, exps, new, pages, q_start):
    """One sequence, K or V.  codes uint8 [pages][128][G][D] and exps int8
    [pages][G] (numpy, changed in place); new float64 [T][G][D]; pages: page of
    each logical block; rows q_start ... q_start + T - 1."""
    T, G = new.shape[:2]
    for kb in range(q_start // BLOCK, (q_start + T - 1) // BLOCK + 1):
        pg = pages[kb]
        r0, r1 = max(q_start - kb * BLOCK, 0), min(q_start + T - kb * BLOCK, BLOCK)
        x = new[kb * BLOCK + r0 - q_start:kb * BLOCK + r1 - q_start]
        for g in range(G):
            a = np.abs(x[:, g])
            fin = a[np.isfinite(a)]
            e = need_exp(fin.max() if fin.size else 0.0)
            if r0 > 0:
                was = int(np.clip(exps[pg, g], MIN_EXP, MAX_EXP))
                e = max(e, was)
                if e > was:
                    codes[pg, :r0, g] = round_e4m3(decode_e4m3(codes[pg, :r0, g]) * 2.0 ** (was - e))
            exps[pg, g] = e
            codes[pg, r0:r1, g] = round_e4m3(x[:, g] * 2.0 ** -e)
