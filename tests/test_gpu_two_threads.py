"""Calls from two host threads at once, each with its stream, workspace and
output: every call succeeds and gives what it gives alone."""
import threading

import pytest
import torch

from tests.test_gpu_cache_q8 import Cache, randq, random_sel
from tests.test_gpu_window import bf16_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def msa():
    assert torch.cuda.is_available()
    import block_sparse_attention_04_gb300 as m
    m.load()
    return m


@pytest.mark.parametrize("call", ["window", "window_q8", "sparse_q8"])
@pytest.mark.parametrize("layouts", [((8, 8), (48, 8)), ((9, 1), (16, 1)), ((4, 2), (12, 2))])
def test_two_head_layouts_of_one_kernel(msa, layouts, call):
    # the streaming kernel's shared memory depends on H / G; both layouts of a
    # pair run the same kernel (heads of a group in one or in two tiles)
    jobs = []
    for i, (H, G) in enumerate(layouts):
        c = Cache([700], G, 128, 6, seed=H)
        q = randq(1, 1, H, 128)
        p = msa.params(1, 1, H, G, 128, 32, 6, kernels="streaming")
        kw = dict(block_table=c.table, num_pool_blocks=c.pages)
        pos = msa.positions([699]), msa.positions([700])
        if call == "sparse_q8":
            sel, ws = random_sel(1, 1, G, [699], 3), msa.q8_workspace(p)

            def run(out, st, p=p, q=q, c=c, sel=sel, ws=ws, kw=kw, pos=pos):
                msa.msa_sparse_attn_q8(p, q, *c.codes, *c.exps, sel, *pos, out, ws, stream=st, **kw)
        else:
            ws = msa.window_workspace(p)
            kv = bf16_cache(c) if call == "window" else (*c.codes, *c.exps)
            fn = msa.msa_window_attn if call == "window" else msa.msa_window_attn_q8

            def run(out, st, p=p, q=q, kv=kv, fn=fn, ws=ws, kw=kw, pos=pos):
                fn(p, 600, 3, q, *kv, *pos, out, ws, stream=st, **kw)
        out = torch.empty_like(q)
        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        run(out, stream.cuda_stream)
        msa.msa_workspace_status(ws, stream)
        jobs.append((run, stream, ws, q, out))
    errors = []
    start = threading.Barrier(2)

    def work(run, stream, ws, q, want):
        try:
            out = torch.empty_like(q)
            torch.cuda.synchronize()
            start.wait(30)
            for _ in range(400):
                run(out, stream.cuda_stream)
            msa.msa_workspace_status(ws, stream)
            if not torch.equal(out, want):
                errors.append("outputs differ")
        except Exception as e:      # a failure of the thread fails the test
            errors.append(repr(e))

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
