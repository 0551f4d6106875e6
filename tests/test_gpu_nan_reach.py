"""A NaN in V of a token that only some queries of a call see: which outputs it
reaches.  Decode kernels: those of the queries that see it.  Prefill kernels:
also, where msa.h says so, outputs of queries near them (a weight of 0 does not
cancel a NaN).  All other outputs are what they are without it."""
import pytest
import torch

from tests.test_gpu_cache_q8 import Cache, randq
from tests.test_gpu_window import bf16_cache

pytestmark = pytest.mark.gpu

H, G, D, DIM = 12, 4, 64, 5            # the NaN sits in dim 5 of KV head 1


@pytest.fixture(scope="module")
def msa():
    assert torch.cuda.is_available()
    import block_sparse_attention_04_gb300 as m
    m.load()
    return m


def with_nan(c, pos, q8):
    """The caches of c with a NaN in V of token `pos` of sequence 0, and those
    with a number there."""
    r = []
    for code in (0x7F, 0x38):
        v = c.codes[1].clone()
        v[c.table[0, pos // 128].long(), pos % 128, 1, DIM] = code
        d = Cache.__new__(Cache)
        d.codes, d.exps = [c.codes[0], v], c.exps
        r.append((*d.codes, *d.exps) if q8 else bf16_cache(d))
    return r


def check(nan_out, out, must, may):
    """nan_out is NaN in (dim, heads of KV head 1) of the queries in `must`, may be
    in those of `may`, and equals `out` everywhere else."""
    hit = nan_out.isnan()
    allowed = torch.zeros_like(hit)
    allowed[0, must | may, 3:6, DIM] = True
    assert not (hit & ~allowed).any()
    assert hit[0, must, 3:6, DIM].all()
    assert torch.isfinite(out).all()
    assert torch.equal(nan_out[~hit], out[~hit])
    return hit


@pytest.mark.parametrize("kernels", ["streaming", "tensorcore"])
@pytest.mark.parametrize("forward", [False, True])
def test_sparse_q8(msa, kernels, forward):
    # 300 queries at 401 ... 700; the NaN at 600, inside block 4 (512 ... 639)
    n, T, nb, pos = 701, 300, 6, 600
    c = Cache([n], G, D, nb, seed=7)
    start = n - T
    q = randq(1, T, H, D)
    t = start + torch.arange(T, device="cuda")
    # every query selects all its causal blocks but every third one leaves block 4 out
    sel = torch.arange(16, device="cuda").expand(1, T, G, 16)
    sel = torch.where(sel <= (t // 128)[None, :, None, None], sel, -1).int()
    skips = (t >= 640) & (t % 3 == 0)
    sel = torch.where((sel == 4) & skips[None, :, None, None], -1, sel).contiguous()
    p = msa.params(1, T, H, G, D, 32, nb, kernels=kernels)
    ws = msa.q8_workspace(p)
    kw = dict(block_table=c.table, num_pool_blocks=c.pages)
    qi = torch.zeros(1, T, G, 32, dtype=torch.bfloat16, device="cuda")
    ki = torch.zeros(c.pages, 128, 32, dtype=torch.bfloat16, device="cuda")
    outs = []
    for kv in with_nan(c, pos, True):
        out = torch.full_like(q, 9.0)
        if forward:      # fewer than 16 blocks: all causal ones are selected
            msa.msa_forward_q8(p, qi, ki, q, *kv, [start], [n], out, ws, **kw)
        else:
            msa.msa_sparse_attn_q8(p, q, *kv, sel, [start], [n], out, ws, **kw)
        msa.msa_workspace_status(ws)
        outs.append(out)
    chosen = torch.ones_like(skips) if forward else ~skips
    must = (t >= pos) & chosen
    none = torch.zeros_like(must)
    may = (t // 128 == pos // 128) & (t < pos) if kernels == "tensorcore" else none
    check(*outs, must, may)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kernels", ["streaming", "tensorcore"])
@pytest.mark.parametrize("sink", [False, True])
def test_window(msa, kernels, q8, sink):
    # 900 queries at 101 ... 1000, a window of 150; the NaN at 400, or at 2, a sink
    # token that all queries see
    n, T, nb, window, pos = 1001, 900, 9, 150, 2 if sink else 400
    c = Cache([n], G, D, nb, seed=9)
    start = n - T
    q = randq(1, T, H, D)
    t = start + torch.arange(T, device="cuda")
    p = msa.params(1, T, H, G, D, 32, nb, kernels=kernels)
    ws = msa.window_workspace(p)
    fn = msa.msa_window_attn_q8 if q8 else msa.msa_window_attn
    outs = []
    for kv in with_nan(c, pos, q8):
        out = torch.full_like(q, 9.0)
        fn(p, window, 3, q, *kv, [start], [n], out, ws, block_table=c.table, num_pool_blocks=c.pages)
        msa.msa_workspace_status(ws)
        outs.append(out)
    must = (t >= pos) & ((t < pos + window) | sink)
    near = (t > pos - 256) & (t < pos + window + 255)
    may = near if kernels == "tensorcore" else torch.zeros_like(must)
    check(*outs, must, may)
