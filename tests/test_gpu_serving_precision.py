"""How near the 8-bit and window attention come to the 64-bit result, with the
rounding that each kernel has and no more.

Element-wise, in the terms of serving_ref: the KV-outer kernels of an 8-bit cache
hold 2^15 p (p at most 1 in its block) and a block's partial sum p code in f16.
Each rounds at 2^-11, so u = 2 * 2^-11; below f16's normal numbers a weight is off
by at most 2^-25 * 2^-15 = 2^-40 of its block's largest, which adds N 2^-40 max|v|,
and a partial by 2^-25 of a code's unit, which adds 16 * 2^-25 * 2^max(ev).  The
streaming and the window kernels hold p in bf16: u = 2^-8.

Norm-wise, e = |got - want| / |want| over all outputs.  An error of bf16 rounding
is uniform within half a step, whose rms is a = 2^-8 / sqrt(3) of the power of two
below the value.  With values m times that power, m in [1, 2), the rms error is
a / sqrt(E m^2) of their rms: 1.48e-3 for m spread evenly (E m^2 = 7 / 3), 1.53e-3
for its logarithm (3 / (2 ln 2)); the rms of the relative errors is a sqrt(E m^-2)
= 1.66e-3 (3 / (8 ln 2)).  V's values are independent of the weights' roundings,
so weights (or partials) with a relative rms error r add r of the norm.  f16 twice:
r = 1.66e-3 / 8 each, e <= sqrt(1.66^2 + 2 (1.66 / 8)^2) 1e-3 = 1.69e-3, where a
rounding to bf16 in the place of one would give at least sqrt(2) 1.48e-3 = 2.09e-3:
the limit is 1.9e-3.  bf16 weights: e <= sqrt(2) 1.66e-3 = 2.35e-3, where one more
rounding to bf16 would give at least sqrt(3) 1.48e-3 = 2.56e-3: the limit is 2.5e-3."""
import pytest
import torch

from tests import serving_ref as sr
from tests.test_gpu_cache_q8 import Cache, randq, random_sel
from tests.test_gpu_window import bf16_cache

pytestmark = pytest.mark.gpu

F16_LIMIT, BF16_LIMIT = 1.9e-3, 2.5e-3


@pytest.fixture(scope="module")
def msa():
    assert torch.cuda.is_available()
    import block_sparse_attention_04_gb300 as m
    m.load()
    return m


def hold(out, want, bound, limit):
    sr.check(out, want, bound)
    e = ((out.double() - want).norm() / want.norm()).item()
    assert e <= limit, "error %.3g of the norm" % e


@pytest.mark.parametrize("kernels", ["streaming", "tensorcore"])
@pytest.mark.parametrize("lens,T,H,G,D,scale", [
    ([5000], 200, 48, 8, 128, None), ([2433, 1130], 130, 10, 2, 64, 0.02),
    ([700, 2600], 64, 16, 1, 128, 0.3), ([900], 400, 4, 4, 64, -0.1)])
def test_sparse_q8(msa, kernels, lens, T, H, G, D, scale):
    B, nb = len(lens), max(-(-n // 128) for n in lens)
    c = Cache(lens, G, D, nb, seed=D + T)
    q = randq(B, T, H, D, seed=B)
    starts = [n - T for n in lens]
    sel = random_sel(B, T, G, starts, 7)
    p = msa.params(B, T, H, G, D, 32, nb, kernels=kernels, scale=scale)
    ws, out = msa.q8_workspace(p), torch.full_like(q, float("nan"))
    msa.msa_sparse_attn_q8(p, q, *c.codes, *c.exps, sel, starts, lens, out, ws,
                           block_table=c.table, num_pool_blocks=c.pages)
    msa.msa_workspace_status(ws)
    k, v = c.values()
    f16 = kernels == "tensorcore"
    want, bound = sr.attend_call(q, k, v, starts, sr.sel_seen(sel, nb * 128, "cuda"),
                                 D ** -0.5 if scale is None else scale,
                                 2 * 2.0 ** -11 if f16 else sr.U_BF16)
    if f16:
        top = max(x.nan_to_num().abs().max().item() for x in v)
        bound = bound + 16 * 128 * 2.0 ** -40 * top + 16 * 2.0 ** (-25 + c.exps[1].max().item())
    hold(out, want, bound, F16_LIMIT if f16 else BF16_LIMIT)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kernels", ["streaming", "tensorcore"])
@pytest.mark.parametrize("lens,T,H,G,D,window,sinks,scale", [
    ([3000], 200, 48, 8, 128, 1000, 5, None), ([2433, 1130], 300, 10, 2, 64, 1 << 20, 0, 0.02),
    ([1500, 700], 33, 16, 1, 128, 300, 130, 0.3)])
def test_window(msa, kernels, q8, lens, T, H, G, D, window, sinks, scale):
    B, nb = len(lens), max(-(-n // 128) for n in lens)
    c = Cache(lens, G, D, nb, seed=D + T + 1)
    q = randq(B, T, H, D, seed=B)
    starts = [n - T for n in lens]
    p = msa.params(B, T, H, G, D, 32, nb, kernels=kernels, scale=scale)
    ws, out = msa.window_workspace(p), torch.full_like(q, float("nan"))
    kv = (*c.codes, *c.exps) if q8 else bf16_cache(c)
    fn = msa.msa_window_attn_q8 if q8 else msa.msa_window_attn
    fn(p, window, sinks, q, *kv, starts, lens, out, ws, block_table=c.table,
       num_pool_blocks=c.pages)
    msa.msa_workspace_status(ws)
    k, v = c.values()
    want, bound = sr.attend_call(q, k, v, starts, sr.window_seen(nb * 128, window, sinks, "cuda"),
                                 D ** -0.5 if scale is None else scale, sr.U_BF16)
    hold(out, want, bound, BF16_LIMIT)
