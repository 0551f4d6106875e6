"""Sparse attention of a (query, group) whose selection holds no token: out is zeros,
lse -inf, the other rows have the bits that they have in any call, and the backward pass
takes such rows as the forward left them."""
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


def case(B, T, H, G, D, starts):
    g = torch.Generator(device="cuda").manual_seed(7)
    mb = (max(starts) + T + 127) // 128

    def bf(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)

    q, k, v = bf(B, T, H, D), bf(B, mb, 128, G, D), bf(B, mb, 128, G, D)
    sel = R.random_sel(T, G, starts, g, "cuda")
    empty = torch.rand(B, T, G, generator=g, device="cuda") < 0.3
    empty[:, -1, 0] = True
    empty[0, 0] = True                      # a query without any
    some = sel.clone()
    some[empty] = -1
    return mb, q, k, v, sel, some, empty


SHAPES = [
    dict(B=1, T=5, H=4, G=2, D=64, starts=[300]),
    dict(B=2, T=1, H=48, G=8, D=128, starts=[0, 2900]),
    dict(B=3, T=70, H=10, G=2, D=64, starts=[0, 51, 2100]),
    dict(B=1, T=600, H=16, G=1, D=128, starts=[1500]),
]


@pytest.mark.parametrize("kernels", ["auto", "streaming", "tensorcore"])
@pytest.mark.parametrize("kw", SHAPES)
def test_forward_and_backward(msa, kw, kernels):
    B, T, H, G, D, starts = (kw[k] for k in ("B", "T", "H", "G", "D", "starts"))
    mb, q, k, v, sel, some, empty = case(**kw)
    kv_len = [s + T for s in starts]
    p = msa.params(B, T, H, G, D, 64, mb, kernels=kernels)
    ws = msa.workspace(p)
    rows = empty.repeat_interleave(H // G, -1)

    def forward(ids, with_lse):
        out = torch.full_like(q, NAN)
        lse = torch.full((B, T, H), NAN, device="cuda")
        if with_lse:
            msa.msa_sparse_attn_lse(p, q, k, v, ids, starts, kv_len, out, lse, ws)
        else:
            msa.msa_sparse_attn(p, q, k, v, ids, starts, kv_len, out, ws)
        msa.msa_workspace_status(ws)
        return out, lse

    full, full_lse = forward(sel, True)
    out, lse = forward(some, True)
    assert (out[rows] == 0).all()
    assert (lse[rows] == -torch.inf).all()
    assert torch.equal(out[~rows], full[~rows]) and torch.equal(lse[~rows], full_lse[~rows])
    assert torch.equal(forward(some, False)[0], out)

    g = torch.Generator(device="cuda").manual_seed(8)
    dout = torch.randn(B, T, H, D, generator=g, device="cuda").to(torch.bfloat16)
    dq, dk, dv = torch.full_like(q, NAN), torch.full_like(k, NAN), torch.full_like(v, NAN)
    bws = msa.sparse_bwd_workspace(p)
    msa.msa_sparse_attn_bwd(p, q, k, v, some, out, lse, dout, starts, kv_len, dq, dk, dv, bws)
    msa.msa_workspace_status(bws)
    want, bound = R.attn_backward(q, k, v, out, dout, starts, kv_len, p.scale, some)
    assert (dq[rows] == 0).all()
    # lse and out are the library's: exponentials within 2^-13 there (a polynomial in a
    # part of them), so that P and dS are too; each gradient by 2^-13 of its terms' size
    R.check(dq, want[0], bound[0] + extra(q, k, v, dout, some, starts, p.scale)[0], "dq")
    _, ek, ev = extra(q, k, v, dout, some, starts, p.scale)
    for b in range(B):
        n = kv_len[b]
        for got, w, e, x, what in ((dk, want[1], bound[1], ek, "dk"), (dv, want[2], bound[2], ev, "dv")):
            flat = [y[b].flatten(0, 1)[:n] for y in (got, w, e, x)]
            R.check(flat[0], flat[1], flat[2] + flat[3], what)


def extra(q, k, v, dout, sel, starts, scale):
    """2^-12 of the sizes of each gradient's terms (P twice in dS: itself and delta)."""
    B, T, H, D = q.shape
    G = k.shape[3]
    eq = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    ek = torch.zeros(k.shape, dtype=torch.float64, device=q.device).flatten(1, 2)
    ev = torch.zeros_like(ek)
    for b in range(B):
        n = starts[b] + T
        for h in range(H):
            g = h // (H // G)
            cnt = R.counts_sel(sel[b, :, g], n, starts[b])
            x, d = q[b, :, h].double(), dout[b, :, h].double()
            y, z = k[b].flatten(0, 1)[:n, g].double(), v[b].flatten(0, 1)[:n, g].double()
            s = torch.where(cnt > 0, x @ y.T * scale, -torch.inf)
            p = torch.nan_to_num(torch.softmax(s, -1), nan=0.0)
            dp = (d @ z.T).abs()
            ds = p * (dp + (p * dp).sum(-1, keepdim=True)) * abs(scale)
            eq[b, :, h] = 2.0 ** -12 * (ds @ y.abs())
            ek[b, :n, g] += 2.0 ** -12 * (ds.T @ x.abs())
            ev[b, :n, g] += 2.0 ** -12 * (p.T @ d.abs())
    return eq, ek.view(k.shape), ev.view(k.shape)


@pytest.mark.parametrize("kernels", ["streaming", "tensorcore"])
def test_ids_out_of_range_alone(msa, kernels):
    """A selection of nothing but ids past the local block: reported, and a row of zeros."""
    kw = SHAPES[0]
    mb, q, k, v, sel, _, _ = case(**kw)
    sel[0, 2, 1] = 77
    p = msa.params(1, 5, 4, 2, 64, 64, mb, kernels=kernels)
    ws = msa.workspace(p)
    out, lse = torch.full_like(q, NAN), torch.full((1, 5, 4), NAN, device="cuda")
    msa.msa_sparse_attn_lse(p, q, k, v, sel, [300], [305], out, lse, ws)
    with pytest.raises(msa.MsaError):
        msa.msa_workspace_status(ws)
    assert (out[0, 2, 2:] == 0).all() and (lse[0, 2, 2:] == -torch.inf).all()
    assert torch.isfinite(out.float()).all()
