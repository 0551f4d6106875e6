"""Failure path of the serving kernels: a pipeline wait that runs out (see
test_gpu_wait_expiry: a poll cap on a correct kernel, no fault and no hang).  It
is recorded as MSA_ERR_TIMEOUT, the kernel drains and exits, and the next call on
the same workspace is exact again.  A poll may suspend its thread for longer than
most waits of these kernels last, so only the cases in SURE must meet an expiry; in the others every status but a timeout or none is an error."""
import pytest
import torch

from tests import serving_ref as sr
from tests.test_gpu_cache_q8 import Cache, random_sel
from tests.test_gpu_window import bf16_cache

pytestmark = pytest.mark.gpu

TIMEOUT = -5
SURE = {"window tensorcore bf16", "window tensorcore bf16 split"}
CASES = {
    # kernels, lens, T, H, G, D, window (None: sparse attention), 8-bit cache
    "window tensorcore bf16": ("tensorcore", [5000, 4000], 300, 12, 4, 128, 2000, False),
    "window tensorcore bf16 split": ("tensorcore", [9000], 20, 12, 4, 128, 9000, False),
    "window tensorcore 8-bit": ("tensorcore", [5000, 4000], 300, 12, 4, 64, 2000, True),
    "window streaming, cluster": ("streaming", [2000], 1, 12, 4, 128, 2000, True),
    "window streaming, runs": ("streaming", [9000] * 6, 1, 48, 8, 128, 9000, True),
    "sparse tensorcore": ("tensorcore", [5000, 4000], 300, 12, 4, 128, None, True),
    "sparse streaming": ("streaming", [5000] * 32, 1, 48, 8, 64, None, True),
}


@pytest.fixture(scope="module")
def msa():
    assert torch.cuda.is_available()
    import block_sparse_attention_04_gb300 as m
    m.load()
    return m


@pytest.mark.parametrize("name", sorted(CASES))
def test_expiry_is_reported_then_the_next_call_is_exact(msa, name):
    kernels, lens, T, H, G, D, window, q8 = CASES[name]
    nb = max(-(-n // 128) for n in lens)
    B = len(lens)
    c = Cache(lens, G, D, nb, seed=61)
    q = torch.randn(B, T, H, D, generator=torch.Generator(device="cuda").manual_seed(62),
                    device="cuda").to(torch.bfloat16)
    starts = [n - T for n in lens]
    p = msa.params(B, T, H, G, D, 32, nb, kernels=kernels)
    paged = dict(block_table=c.table, num_pool_blocks=c.pages)
    out = torch.empty_like(q)
    kv = (*c.codes, *c.exps) if q8 else bf16_cache(c)
    if window is None:
        sel, ws = random_sel(B, T, G, starts, 63), msa.q8_workspace(p)
        seen = sr.sel_seen(sel, nb * 128, "cuda")

        def call():
            msa.msa_sparse_attn_q8(p, q, *kv, sel, starts, lens, out, ws, **paged)
    else:
        ws = msa.window_workspace(p)
        seen = sr.window_seen(nb * 128, window, 0, "cuda")

        def call():
            fn = msa.msa_window_attn_q8 if q8 else msa.msa_window_attn
            fn(p, window, 0, q, *kv, starts, lens, out, ws, **paged)

    def status():
        try:
            msa.msa_workspace_status(ws)
            return 0
        except msa.MsaError as e:
            return e.status

    found = []
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")   # larger than L2
    try:
        msa.msa_debug_set_wait_polls(1)
        for i in range(4):
            flush.fill_(i)
            call()
            found.append(status())
    finally:
        msa.msa_debug_set_wait_polls(0)
    torch.cuda.synchronize()              # the context is still usable
    assert set(found) <= {0, TIMEOUT} and (TIMEOUT in found or name not in SURE), found
    out.fill_(float("nan"))
    call()
    assert status() == 0
    k, v = c.values()
    want, bound = sr.attend_call(q, k, v, starts, seen, D ** -0.5, 2 * sr.U_BF16)
    sr.check(out, want, bound)
