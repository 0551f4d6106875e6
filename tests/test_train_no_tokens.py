"""The training pass called with tensors of no tokens (T = 0): accepted, nothing is read
or written.  Such a call returns before it touches a device, so no GPU is needed."""
import pytest
import torch

import block_sparse_attention_04_gb300 as msa
from block_sparse_attention_04_gb300 import _build

H, G, D, MB = 4, 2, 64, 3


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return msa.load()


def bf(*shape):
    return torch.full(shape, 3.0, dtype=torch.bfloat16)


def scratch(n):
    x = torch.zeros(n + 256, dtype=torch.uint8)
    return x[-x.data_ptr() % 256:][:n]


def aligned(*shape, dtype=torch.bfloat16):
    n = torch.Size(shape).numel() * torch.empty(0, dtype=dtype).element_size()
    x = scratch(n).view(dtype).view(shape)
    x.fill_(3.0)
    return x


@pytest.mark.parametrize("B", [1, 2])
@pytest.mark.parametrize("fused", [False, True])
def test_rope(B, fused):
    p, r = msa.params(B, 0, H, G, D, 32, MB), msa.rope(64)
    starts = [5 * b for b in range(B)]

    def rows():
        if fused:
            return bf(B, 0, H + 2 * G, D).split([H, G, G], 2)
        return bf(B, 0, H, D), bf(B, 0, G, D), bf(B, 0, G, D)

    w = aligned(D)
    caches = [aligned(B, MB, 128, G, D) for _ in range(2)]
    idx = aligned(B, MB, 128, 32)
    weights = [aligned(D, dtype=torch.float32) for _ in range(2)]
    msa.msa_rope_append(p, r, *rows(), bf(B, 0, 32), w, w, starts, bf(B, 0, H, D), *caches, idx,
                        scratch(256), stream=0)
    msa.msa_rope_append(p, r, *rows(), None, None, None, starts, bf(B, 0, H, D), *caches, None,
                        scratch(256), stream=0)
    q, k, _ = rows()
    ws = scratch(msa.msa_rope_append_bwd_workspace_bytes(p))
    msa.msa_rope_append_bwd(p, r, q, k, w, w, starts, bf(B, 0, H, D), *caches, *rows(), *weights, ws,
                            stream=0)
    assert all((x == 3).all() for x in (*caches, idx, *weights, w))


@pytest.mark.parametrize("B", [1, 2])
def test_attention(B):
    p = msa.params(B, 0, H, G, D, 32, MB)
    starts = lens = [5 * b for b in range(B)]
    q, out, dout, dq = (bf(B, 0, H, D) for _ in range(4))
    lse = torch.empty(B, 0, H)
    sel = torch.empty(B, 0, G, 16, dtype=torch.int32)
    k, v, dk, dv = (aligned(B, MB, 128, G, D) for _ in range(4))
    ws = scratch(1 << 20)
    msa.msa_dense_attn_lse(p, q, k, v, starts, lens, out, lse, ws, stream=0)
    big = scratch(msa.msa_workspace_bytes(p))
    msa.msa_sparse_attn_lse(p, q, k, v, sel, starts, lens, out, lse, big, stream=0)
    big = scratch(max(msa.msa_dense_bwd_workspace_bytes(p), msa.msa_sparse_bwd_workspace_bytes(p)))
    msa.msa_dense_attn_bwd(p, q, k, v, out, lse, dout, starts, lens, dq, dk, dv, big, stream=0)
    msa.msa_sparse_attn_bwd(p, q, k, v, sel, out, lse, dout, starts, lens, dq, dk, dv, big, stream=0)
    assert all((x == 3).all() for x in (k, v, dk, dv))


def test_what_is_still_refused():
    """Without tokens: a null address, other shapes, a missing cache.  With tokens: an array
    without elements."""
    p, r = msa.params(2, 0, H, G, D, 32, MB), msa.rope(64)
    w, cache = aligned(D), aligned(2, MB, 128, G, D)
    rows = bf(2, 0, H, D), bf(2, 0, G, D), bf(2, 0, G, D)

    def go(p, q, k, v, k_cache=cache):
        msa.msa_rope_append(p, r, q, k, v, None, w, w, [0, 0], aligned(2, 1, H, D), k_cache, cache,
                            None, scratch(256), stream=0)
    go(p, *rows)
    for bad in (0, None):
        with pytest.raises(msa.MsaError):
            go(p, bad, *rows[1:])
    with pytest.raises(msa.MsaError):
        go(p, *rows, k_cache=None)
    for bad in (bf(2, 0, H, D // 2), bf(1, 0, H, D), bf(2, 1, H, D)):
        with pytest.raises(ValueError):
            go(p, bad, *rows[1:])
    one = msa.params(2, 1, H, G, D, 32, MB)
    with pytest.raises(ValueError):
        go(one, *rows)
    with pytest.raises(msa.MsaError):
        msa.msa_dense_attn_lse(one, bf(2, 0, H, D), cache, cache, [0, 0], [1, 1], bf(2, 0, H, D),
                               torch.empty(2, 0, H), scratch(1 << 24), stream=0)
