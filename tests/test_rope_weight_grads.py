"""The norm weights' gradients of msa_rope_append_bwd under a bound of the kernel's real
depth, which rejects a lost or doubled share of one CTA.

dw_d = sum over tokens and heads of dn_d x_d r.  A term is off by 2^-20 A |x| r through dn
(A the size of its pair) and (D + 32) 2^-24 of its size through r (a sum of D squares, a
reciprocal root) and its products.  It is then summed in fp32, one after another within a
thread (five rows of every token of its CTA), over at most four lanes, four warps, each
32nd CTA and the 32 sums of those:
  depth = 5 tokens + 2 + 4 + ctas / 32 + 1 + 32,
  |dw - exact| <= (2^-20 + (D + 32 + depth) 2^-24) (1 + 2^-10) sum A |x| r."""
import pytest
import torch

from tests import train_ref as R

SMS, CTAS_PER_SM, ROWS_EACH, THREADS = 152, 4, 5, 128


def depth(B, T, H, G, D):
    """Terms that a sum passes through one after another, at most."""
    n, resident, heads, rows = B * T, SMS * CTAS_PER_SM, H + 2 * G, THREADS // (D // 8)
    least, most = -(-heads // (rows * ROWS_EACH)), -(-heads // rows)
    parts = max(min(resident // n if n < resident else 1, most), least)
    runs = min(max(resident // parts, 1), n)
    return ROWS_EACH * -(-n // runs) + 2 + 4 + -(-runs * parts // 32) + 1 + 32


def terms(x, w, dy, t, freqs, interleaved, mscale, eps):
    """dn x r and A |x| r of every row, float64."""
    dy, x = dy.double(), x.double()
    dn = R.rotate(dy, t, freqs, interleaved, mscale, -1.0)
    A = R.pair_size(dy, 2 * len(freqs), interleaved, mscale)
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return dn * n, A * n.abs()


def weight_bound(sizes, D, d):
    return (2.0 ** -20 + (D + 32 + d) * 2.0 ** -24) * (1 + 2.0 ** -10) * sizes.sum(dim=(0, 1, 2))


SHAPES = [
    dict(B=5, T=1001, H=48, G=8, D=128, rot=96, interleaved=False),
    dict(B=1, T=3000, H=12, G=4, D=128, rot=128, interleaved=True),
    dict(B=3, T=700, H=64, G=4, D=64, rot=16, interleaved=False),
]


@pytest.mark.parametrize("kw", SHAPES)
def test_the_bound_rejects_a_lost_share(kw):
    """No sum at all, and the sums without (or with twice) one CTA's tokens, are outside."""
    B, T, H, G, D, rot = (kw[k] for k in ("B", "T", "H", "G", "D", "rot"))
    g = torch.Generator().manual_seed(1)
    x, dy = (torch.randn(B, T, H, D, generator=g).to(torch.bfloat16) for _ in range(2))
    t = torch.arange(T).expand(B, T)
    freqs = [10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]
    each, sizes = terms(x, None, dy, t, freqs, kw["interleaved"], 1.0, 1e-6)
    want = each.sum(dim=(0, 1, 2))
    bound = weight_bound(sizes, D, depth(B, T, H, G, D))
    assert (want.abs() > bound).float().mean() > 0.9
    # the fewest rows that a CTA of this grid sums: every resident-th token, a part of its heads
    runs = SMS * CTAS_PER_SM // max(1, -(-(H + 2 * G) // (ROWS_EACH * (THREADS // (D // 8)))))
    share = each.reshape(B * T, H, D)[::runs, :max(1, H // 4)].sum(dim=(0, 1))
    assert (share.abs() > bound).float().mean() > 0.3
    with pytest.raises(AssertionError):
        R.check(want - share, want, bound)
    with pytest.raises(AssertionError):
        R.check(torch.zeros_like(want), want, bound)


@pytest.mark.gpu
@pytest.mark.parametrize("kw", SHAPES + [
    dict(B=1, T=1, H=4, G=1, D=64, rot=64, interleaved=False),
    dict(B=64, T=1, H=48, G=8, D=128, rot=64, interleaved=False),
    dict(B=2, T=301, H=128, G=8, D=128, rot=128, interleaved=False),
    dict(B=7, T=1009, H=7, G=7, D=64, rot=32, interleaved=True)])
def test_weight_gradients(kw):
    import block_sparse_attention_04_gb300 as msa
    from tests.test_gpu_rope import Case, run_bwd
    B, T, H, G, D = (kw[k] for k in ("B", "T", "H", "G", "D"))
    c = Case(Di=64, starts=[3 * b for b in range(B)], **kw)
    ws, r = run_bwd(msa, c)
    msa.msa_workspace_status(ws)
    args = (c.t, c.freqs(r), c.interleaved, 1.0, 1e-6)
    rows = c.dkc.view(B, -1, G, D)[c.own].view(B, T, G, D)
    for x, w, dy, got, what in ((c.q, c.qw, c.dqo, c.dqw, "dq_weight"),
                                (c.k, c.kw, rows, c.dkw, "dk_weight")):
        each, sizes = terms(x, w, dy, *args)
        R.check(got, each.sum(dim=(0, 1, 2)), weight_bound(sizes, D, depth(B, T, H, G, D)), what)
