"""The sparse backward pass reports an id past the local block whatever the workspace held
before, and a call without one is not taken for one that has."""
import pytest
import torch

from tests import train_ref as R

pytestmark = pytest.mark.gpu


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


@pytest.mark.parametrize("T", [3, 500, 9000])        # 9000 rows: two passes
@pytest.mark.parametrize("early", [False, True])     # with the first positions' statistics
def test_reported_in_every_state(msa, T, early):
    H, G, D = 2, 2, 64
    start = 0 if early else 400
    g = torch.Generator(device="cuda").manual_seed(3)
    mb = (start + T + 127) // 128
    bf = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)   # noqa: E731
    q, dout = bf(1, T, H, D), bf(1, T, H, D)
    k, v = bf(1, mb, 128, G, D), bf(1, mb, 128, G, D)
    sel = R.random_sel(T, G, [start], g, "cuda")
    p = msa.params(1, T, H, G, D, 64, mb)
    out, lse = torch.empty_like(q), torch.empty(1, T, H, device="cuda")
    msa.msa_sparse_attn_lse(p, q, k, v, sel, [start], [start + T], out, lse, msa.workspace(p))
    grads = [torch.empty_like(x) for x in (q, k, v)]
    ws = msa.sparse_bwd_workspace(p)
    for at in (0, T - 1):
        bad = sel.clone()
        bad[0, at, G - 1, 15] = (start + at) // 128 + 1
        for fill in (0, 1, 2, 3, 0xFF):
            for ids, want in ((sel, 0), (bad, -1), (bad, -1), (sel, 0)):
                ws[:256] = fill
                msa.msa_sparse_attn_bwd(p, q, k, v, ids, out, lse, dout, [start], [start + T], *grads,
                                        ws)
                assert status(msa, ws) == want
