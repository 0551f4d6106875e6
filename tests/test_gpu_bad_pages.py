"""Table entries outside the pool in attention calls: reported, never read, and
attended to as tokens whose K and V are zero, by both kernel families."""
import pytest
import torch

from tests import serving_ref as sr
from tests.test_gpu_cache_q8 import Cache, randq, random_sel
from tests.test_gpu_window import bf16_cache

pytestmark = pytest.mark.gpu

KERNELS = ["streaming", "tensorcore", "auto"]


@pytest.fixture(scope="module")
def msa():
    assert torch.cuda.is_available()
    import block_sparse_attention_04_gb300 as m
    m.load()
    return m


def holed(c, bad):
    """c's values with the blocks (b, kb) of `bad` as zeros, and its table with
    entries outside the pool there."""
    k, v = c.values()
    table = c.table.clone()
    for (b, kb), entry in bad.items():
        table[b, kb] = entry
        for x in (k, v):
            x[b] = x[b].clone()
            x[b][kb * 128:(kb + 1) * 128] = 0
    return k, v, table


def reported(msa, ws):
    with pytest.raises(msa.MsaError) as e:
        msa.msa_workspace_status(ws)
    assert e.value.status == -1


@pytest.mark.parametrize("kernels", KERNELS)
@pytest.mark.parametrize("T,H,G,D", [(1, 48, 8, 128), (2, 12, 4, 64), (150, 12, 4, 128), (40, 16, 1, 64)])
def test_sparse_q8(msa, kernels, T, H, G, D):
    lens, nb = [1500, 900], 13
    c = Cache(lens, G, D, nb, seed=T)
    starts = [n - T for n in lens]
    last = (lens[1] - 1) // 128
    k, v, table = holed(c, {(0, 3): -1, (0, 10): c.pages, (1, last): 1 << 30, (1, 0): -(1 << 31)})
    q, sel = randq(2, T, H, D), random_sel(2, T, G, starts, 5)
    p = msa.params(2, T, H, G, D, 32, nb, kernels=kernels)
    ws, out = msa.q8_workspace(p), torch.full_like(q, float("nan"))
    msa.msa_sparse_attn_q8(p, q, *c.codes, *c.exps, sel, starts, lens, out, ws, block_table=table,
                           num_pool_blocks=c.pages)
    reported(msa, ws)
    want, bound = sr.attend_call(q, k, v, starts, sr.sel_seen(sel, nb * 128, "cuda"), D ** -0.5,
                                 2 * sr.U_BF16)
    sr.check(out, want, bound)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kernels", KERNELS)
@pytest.mark.parametrize("T,H,G,D,window", [(1, 48, 8, 128, 1 << 20), (3, 10, 2, 64, 500),
                                            (300, 12, 4, 128, 700), (20, 16, 1, 64, 1 << 20)])
def test_window(msa, kernels, T, H, G, D, window, q8):
    lens, nb = [1500, 900], 13
    c = Cache(lens, G, D, nb, seed=T + 1)
    starts = [n - T for n in lens]
    last = (lens[1] - 1) // 128
    k, v, table = holed(c, {(0, 0): -1, (0, 9): c.pages, (1, last): 1 << 30, (1, 5): -7})
    q = randq(2, T, H, D)
    p = msa.params(2, T, H, G, D, 32, nb, kernels=kernels)
    ws, out = msa.window_workspace(p), torch.full_like(q, float("nan"))
    kv = (*c.codes, *c.exps) if q8 else bf16_cache(c)
    fn = msa.msa_window_attn_q8 if q8 else msa.msa_window_attn
    fn(p, window, 2, q, *kv, starts, lens, out, ws, block_table=table, num_pool_blocks=c.pages)
    reported(msa, ws)
    want, bound = sr.attend_call(q, k, v, starts, sr.window_seen(nb * 128, window, 2, "cuda"),
                                 D ** -0.5, sr.U_BF16)
    sr.check(out, want, bound)
