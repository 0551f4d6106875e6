"""Failure path of the attention's backward pass, each kind of CTA for itself: a copy that
a test delays, and waits that give up after one poll.  The call has to report the expiry,
drain what it issued and leave the context and the workspace usable; the next call, without
the cap, is right again.  Everything that is waited for would have come."""
import pytest
import torch

from tests import train_ref as R

pytestmark = pytest.mark.gpu
NAN = float("nan")
KV, DQ = 1, 2


@pytest.fixture(scope="module")
def msa():
    assert torch.cuda.is_available()
    import block_sparse_attention_04_gb300 as m
    m.load()
    return m


def status(msa, ws):
    try:
        msa.msa_workspace_status(ws)
        return 0
    except msa.MsaError as e:
        return e.status


@pytest.mark.parametrize("sparse,kind,at", [
    (True, KV, 0), (True, KV, 1), (True, KV, 2), (True, KV, 7),    # rows of a unit's tiles
    (False, KV, 0), (False, KV, 1),                                # K and V of a unit
    (False, DQ, 0), (False, DQ, 1), (False, DQ, 6)])               # K of a block
@pytest.mark.parametrize("D", [64, 128])
def test_expiry_is_reported_then_next_call_is_exact(msa, D, sparse, kind, at):
    B, T, H, G, starts = 2, 1500, 16, 8, [300, 0]
    g = torch.Generator(device="cuda").manual_seed(4)
    mb = 15
    bf = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)   # noqa: E731
    q, dout = bf(B, T, H, D), bf(B, T, H, D)
    k, v = bf(B, mb, 128, G, D), bf(B, mb, 128, G, D)
    lens = [s + T for s in starts]
    sel = R.random_sel(T, G, starts, g, "cuda") if sparse else None
    p = msa.params(B, T, H, G, D, 64, mb)
    out, lse = R.attn_forward(q, k, v, starts, p.scale, sel)
    grads = [torch.full_like(x, NAN) for x in (q, k, v)]
    ws = msa.sparse_bwd_workspace(p) if sparse else msa.dense_bwd_workspace(p)
    ws.fill_(0xFF)

    def call():
        for x in grads:
            x.fill_(NAN)
        fn = msa.msa_sparse_attn_bwd if sparse else msa.msa_dense_attn_bwd
        fn(p, q, k, v, *((sel,) if sparse else ()), out, lse, dout, starts, lens, *grads, ws)
        return status(msa, ws)

    assert call() == 0
    first = [torch.nan_to_num(x) for x in grads]
    try:
        # the delay alone is waited for
        msa.msa_debug_delay_copies(kind, at, 500)
        assert call() == 0
        assert all(torch.equal(a, torch.nan_to_num(b)) for a, b in zip(first, grads))
        msa.msa_debug_delay_copies(kind, at, 5000)
        msa.msa_debug_set_wait_polls(1)
        assert [call() for _ in range(3)] == [-5] * 3
    finally:
        msa.msa_debug_set_wait_polls(0)
        msa.msa_debug_delay_copies(0, 0, 0)
    torch.cuda.synchronize()
    for _ in range(2):
        assert call() == 0
        assert all(torch.equal(a, torch.nan_to_num(b)) for a, b in zip(first, grads))
    want, bound = R.attn_backward(q, k, v, out, dout, starts, lens, p.scale, sel)
    R.check(grads[0], want[0], bound[0], "dq")
    for b in range(B):
        for i in (1, 2):
            R.check(*(x[b].flatten(0, 1)[:lens[b]] for x in (grads[i], want[i], bound[i])), "dk, dv")
