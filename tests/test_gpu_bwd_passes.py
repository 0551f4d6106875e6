"""Sparse backward calls of three and more passes (8192 query rows each): a middle pass
adds to the running sums and hands them on.  Blocks are met in every way: in all passes,
in the first and the last alone, in a middle one alone, never, in several pieces in one
pass and in one piece in another."""
import pytest
import torch

from tests import train_ref as R

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module")
def msa():
    assert torch.cuda.is_available()
    import block_sparse_attention_04_gb300 as m
    m.load()
    return m


def selection(B, T, G, starts, per, g):
    """Which ids a query may choose depends on its pass: block 0 in all (by every query of
    the second), 1 in the first and last, 2 in the second alone, 3 never, the others by
    chance; lb where it is not one of those.  [B][T][G][16]"""
    sel = R.random_sel(T, G, starts, g, "cuda")
    i = torch.arange(T, device="cuda")[None, :, None, None]
    n, last = i // per, (T - 1) // per
    keep = ((sel == 1) & ((n == 0) | (n == last))) | ((sel == 2) & (n == 1)) | (sel >= 4) | (sel == 0)
    sel = torch.where(keep, sel, -1)
    some = torch.rand(B, T, G, 1, generator=g, device="cuda") < 0.25
    first = torch.where(some | (n == 1), 0, -1).expand(B, T, G, 1)
    sel = torch.where(sel == 0, -1, sel)
    free = (sel < 0).int().argmax(-1, keepdim=True)       # a free slot, if there is one
    return torch.where((torch.arange(16, device="cuda") == free) & (sel < 0), first,
                       sel).int().contiguous()


@pytest.mark.parametrize("kw", [
    dict(B=8, T=3300, H=2, G=1, D=64, starts=[0, 1, 127, 128, 129, 500, 640, 0]),     # 4 passes
    dict(B=8, T=2100, H=16, G=1, D=128, starts=[0, 64, 128, 0, 700, 3, 5, 900]),      # 3
    dict(B=16, T=1700, H=6, G=2, D=128, starts=[97 * b for b in range(16)])])         # 4
def test_middle_passes(msa, kw):
    B, T, H, G, D, starts = (kw[k] for k in ("B", "T", "H", "G", "D", "starts"))
    g = torch.Generator(device="cuda").manual_seed(11)
    more = 300                                            # tokens behind the last query
    lens = [s + T + more for s in starts]
    mb = (max(lens) + 127) // 128 + 1
    bf = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)   # noqa: E731
    q, dout = bf(B, T, H, D), bf(B, T, H, D)
    k, v = bf(B, mb, 128, G, D), bf(B, mb, 128, G, D)
    per = 8192 // B
    assert T > 2 * per
    sel = selection(B, T, G, starts, per, g)
    n = torch.arange(T, device="cuda")[None, :, None, None] // per
    has = lambda kb: [bool((sel == kb)[(n == x).expand_as(sel)].any())               # noqa: E731
                      for x in range((T - 1) // per + 1)]
    assert all(has(0)) and not any(has(3))
    assert has(1)[0] and has(1)[-1] and not any(has(1)[1:-1])
    assert has(2)[1] and sum(has(2)) == 1
    p = msa.params(B, T, H, G, D, 64, mb)
    out, lse = R.attn_forward(q, k, v, starts, p.scale, sel)
    grads = [torch.full_like(x, NAN) for x in (q, k, v)]
    ws = msa.sparse_bwd_workspace(p)
    ws.fill_(0xFF)                                        # running sums: NaN
    msa.msa_sparse_attn_bwd(p, q, k, v, sel, out, lse, dout, starts, lens, *grads, ws)
    msa.msa_workspace_status(ws)
    want, bound = R.attn_backward(q, k, v, out, dout, starts, lens, p.scale, sel)
    R.check(grads[0], want[0], bound[0], "dq")
    for b in range(B):
        for i, what in ((1, "dk"), (2, "dv")):
            x, w, e = (y[b].flatten(0, 1) for y in (grads[i], want[i], bound[i]))
            R.check(x[:lens[b]], w[:lens[b]], e[:lens[b]], what)
            assert (x[starts[b] + T:lens[b]] == 0).all() and (x[3 * 128:4 * 128] == 0).all()
            assert torch.isnan(x[lens[b]:].float()).all()
    again = [x.clone() for x in grads]
    msa.msa_sparse_attn_bwd(p, q, k, v, sel, out, lse, dout, starts, lens, *grads, ws)
    assert all(torch.equal(torch.nan_to_num(a), torch.nan_to_num(b)) for a, b in zip(again, grads))
