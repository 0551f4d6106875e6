"""Sizes of the serving operators that the other tests leave out: every number of
query heads per KV head, prefill calls of more rows than a pass holds, and page
operations over many rows and long ones."""
import numpy as np
import pytest
import torch

from tests import serving_ref as sr
from tests.test_gpu_cache_q8 import Cache, randq, random_sel
from tests.test_gpu_pages import World, contiguous_world
from tests.test_gpu_window import bf16_cache

pytestmark = pytest.mark.gpu

KERNELS = ["streaming", "tensorcore"]


@pytest.fixture(scope="module")
def msa():
    assert torch.cuda.is_available()
    import block_sparse_attention_04_gb300 as m
    m.load()
    return m


def sparse(msa, c, q, sel, starts, lens, nb, kernels):
    B, T, H, D = q.shape
    p = msa.params(B, T, H, c.codes[0].shape[2], D, 32, nb, kernels=kernels)
    ws, out = msa.q8_workspace(p), torch.full_like(q, float("nan"))
    msa.msa_sparse_attn_q8(p, q, *c.codes, *c.exps, sel, starts, lens, out, ws,
                           block_table=c.table, num_pool_blocks=c.pages)
    msa.msa_workspace_status(ws)
    return out


@pytest.mark.parametrize("kernels", KERNELS)
@pytest.mark.parametrize("hpg", range(1, 17))
@pytest.mark.parametrize("T,D", [(3, 128), (70, 64)])
def test_heads_per_group(msa, kernels, hpg, T, D):
    lens, G, nb = [900, 431], 2, 8
    c = Cache(lens, G, D, nb, seed=hpg)
    q = randq(2, T, hpg * G, D, seed=hpg)
    starts = [n - T for n in lens]
    k, v = c.values()
    sel = random_sel(2, T, G, starts, hpg)
    out = sparse(msa, c, q, sel, starts, lens, nb, kernels)
    u = sr.U_BF16 if kernels == "streaming" else 2 * 2.0 ** -11 + 2.0 ** -20
    want, bound = sr.attend_call(q, k, v, starts, sr.sel_seen(sel, nb * 128, "cuda"), D ** -0.5, u)
    sr.check(out, want, bound)
    want, bound = sr.attend_call(q, k, v, starts, sr.window_seen(nb * 128, 300, 5, "cuda"),
                                 D ** -0.5, sr.U_BF16)
    p = msa.params(2, T, hpg * G, G, D, 32, nb, kernels=kernels)
    ws = msa.window_workspace(p)
    kw = dict(block_table=c.table, num_pool_blocks=c.pages)
    for fn, kv in ((msa.msa_window_attn_q8, (*c.codes, *c.exps)),
                   (msa.msa_window_attn, bf16_cache(c))):
        out = torch.full_like(q, float("nan"))
        fn(p, 300, 5, q, *kv, starts, lens, out, ws, **kw)
        msa.msa_workspace_status(ws)
        sr.check(out, want, bound)


@pytest.mark.parametrize("kernels", KERNELS)
@pytest.mark.parametrize("lens,T", [([9001], 9001), ([3000, 2999, 2901], 2900)])
def test_prefill_of_more_rows_than_a_pass(msa, kernels, lens, T):
    # passes of 8192 (sequence, query) rows on tensor cores, of 2048 streaming
    B, H, G, D, nb = len(lens), 2, 1, 64, -(-max(lens) // 128)
    c = Cache(lens, G, D, nb, seed=T)
    q = randq(B, T, H, D, seed=T)
    starts = [n - T for n in lens]
    sel = random_sel(B, T, G, starts, T)
    out = sparse(msa, c, q, sel, starts, lens, nb, kernels)
    k, v = c.values()
    u = sr.U_BF16 if kernels == "streaming" else 2 * 2.0 ** -11 + 2.0 ** -20
    want, bound = sr.attend_call(q, k, v, starts, sr.sel_seen(sel, nb * 128, "cuda"), D ** -0.5, u)
    sr.check(out, want, bound)


@pytest.mark.parametrize("rows,mb,span", [(256, 9, 1), (256, 40, 33), (3, 9000, 8300)])
def test_alloc_and_free_over_many_rows_and_long_ones(msa, rows, mb, span):
    pages = 20000
    w = World(pages, rows, mb, rows, fill=0.0)
    taken = w.rng.permutation(pages)[:pages // 4]
    w.refs[taken] = 1                          # pages of other tables
    w.pools = w.pools[3:]
    w.device(msa)
    ids = w.rng.permutation(rows).tolist()
    first = w.rng.integers(0, mb - span + 1, rows).tolist()
    last = [a + span for a in first]
    free = np.flatnonzero(w.refs == 0)
    need = rows * span
    msa.msa_pages_alloc(pages, w.d_table, w.d_refs, ids, first, last, w.ws)
    if need <= len(free):
        msa.msa_workspace_status(w.ws)
    else:
        with pytest.raises(msa.MsaError):
            msa.msa_workspace_status(w.ws)
    give = iter(free)
    for r, a, z in zip(ids, first, last):
        for kb in range(a, z):
            w.table[r, kb] = next(give, -1)
    w.refs[w.table[w.table >= 0]] = 1
    w.same()
    half = [a + span // 2 for a in first]
    msa.msa_pages_free(pages, w.d_table, w.d_refs, ids, half, last, w.ws)
    msa.msa_workspace_status(w.ws)
    w.free(ids, half, last)
    w.same()


def test_fork_of_256_rows_of_one_prompt(msa):
    lens = [128 * 20 + 77] + [0] * 256
    w = contiguous_world(400, 257, 21, lens, seed=3)
    w.device(msa)
    src, dst, n = [0] * 256, list(range(1, 257)), [lens[0] - (i % 3) for i in range(256)]
    msa.msa_pages_fork(w.set, 400, w.d_table, w.d_refs, src, dst, n, w.ws)
    msa.msa_workspace_status(w.ws)
    w.fork(src, dst, n)
    w.same()
