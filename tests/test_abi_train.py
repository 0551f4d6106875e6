"""C-ABI checks of the training pass that need no GPU: argument refusals on the host,
and the binding's checks of strides."""
import ctypes

import pytest
import torch

import block_sparse_attention_04_gb300 as msa
from block_sparse_attention_04_gb300 import _build

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
PTR, BIG = 0x100000, 1 << 40


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return msa.load()


def P(**kw):
    base = dict(B=2, T=0, H=48, G=8, D=128, Di=64, max_blocks=16)
    base.update(kw)
    return msa.params(**base)


def i32(*x):
    return (ctypes.c_int32 * len(x))(*x)


def rope_append(lib, p=None, r=None, table=None, pool=0, rows=None, strides=None, weights=(PTR, PTR),
                kidx=PTR, q_start=(0, 0), outs=None, ws=PTR, ws_bytes=BIG, no_p=False, no_r=False):
    p = p or P()
    r = r or msa.rope(64)
    rows = [PTR] * 3 if rows is None else rows
    strides = [64 * 128, 8 * 128, 8 * 128] if strides is None else strides
    outs = [PTR] * 4 if outs is None else outs
    return lib.msa_rope_append(None if no_p else ctypes.byref(p), None if no_r else ctypes.byref(r),
                               table, pool, *rows, *strides, *weights, kidx,
                               None if q_start is None else i32(*q_start), *outs, ws, ws_bytes, None)


def test_rope_append_refusals(lib):
    go = lambda **kw: rope_append(lib, **kw)          # noqa: E731
    assert go() == OK
    assert go(no_p=True) == INVALID and go(no_r=True) == INVALID
    assert go(p=P(D=96)) == UNSUPPORTED
    assert go(table=PTR, pool=0) == INVALID and go(table=PTR, pool=4) == OK
    assert go(q_start=None) == INVALID and go(q_start=(-1, 0)) == INVALID
    assert go(p=P(T=9), q_start=(0, 16 * 128 - 8)) == INVALID
    for i in range(3):
        assert go(rows=[PTR] * i + [None] + [PTR] * (2 - i)) == INVALID
        assert go(rows=[PTR] * i + [PTR + 8] + [PTR] * (2 - i)) == INVALID
        for s in (8, 48 * 128 + 4 if i == 0 else 8 * 128 + 4, 0, -8192):
            good = [64 * 128, 8 * 128, 8 * 128]
            good[i] = s
            assert go(strides=good) == INVALID
    for i in range(4):
        assert go(outs=[PTR] * i + [None] + [PTR] * (3 - i)) == INVALID
        assert go(outs=[PTR] * i + [PTR + 4] + [PTR] * (3 - i)) == INVALID
    assert go(kidx=None, outs=[PTR] * 3 + [None]) == OK
    assert go(weights=(None, None)) == OK and go(weights=(None, PTR + 2)) == INVALID
    assert go(ws=None) == INVALID and go(ws=PTR + 16) == INVALID and go(ws_bytes=255) == WORKSPACE


def test_rope_parameters(lib):
    def go(p=None, **kw):
        r = msa.rope(64)
        for k, v in kw.items():
            if k == "freq":
                r.inv_freq[3] = v
            else:
                setattr(r, k, v)
        return rope_append(lib, p=p, r=r)
    for rot, want in [(0, OK), (16, OK), (128, OK), (144, INVALID), (-16, INVALID), (24, UNSUPPORTED),
                      (1, UNSUPPORTED)]:
        assert go(rot=rot) == want
    assert go(p=P(D=64, H=8, G=1), rot=80) == INVALID
    assert go(interleaved=2) == INVALID and go(interleaved=1) == OK
    for bad in (float("nan"), float("inf"), -1e-6):
        assert go(eps=bad) == INVALID
    assert go(eps=0.0) == OK
    for bad in (float("nan"), float("inf")):
        assert go(mscale=bad) == INVALID and go(freq=bad) == INVALID


def test_rope_append_bwd_refusals(lib):
    need = lib.msa_rope_append_bwd_workspace_bytes(ctypes.byref(P()))
    assert need > 0 and lib.msa_rope_append_bwd_workspace_bytes(ctypes.byref(P(H=47))) == 0

    def go(p=None, x=(PTR, PTR), xs=(6144, 1024), w=(PTR, PTR), q_start=(0, 0), grads=(PTR,) * 6,
           gs=(6144, 1024, 1024), dw=(PTR, PTR), ws=PTR, ws_bytes=need):
        p = p or P()
        return lib.msa_rope_append_bwd(ctypes.byref(p), ctypes.byref(msa.rope(128)), *x, *xs, *w,
                                       None if q_start is None else i32(*q_start), *grads, *gs, *dw, ws,
                                       ws_bytes, None)
    assert go() == OK
    assert go(q_start=None) == INVALID and go(p=P(T=9), q_start=(2040, 0)) == INVALID
    for i in range(6):
        for bad in (None, PTR + 8):
            assert go(grads=[PTR] * i + [bad] + [PTR] * (5 - i)) == INVALID
    for i in range(3):
        gs = [6144, 1024, 1024]
        gs[i] -= 8
        assert go(gs=gs) == INVALID
    assert go(x=(None, PTR)) == INVALID and go(x=(PTR, None)) == INVALID
    assert go(x=(None, PTR), xs=(0, 1024), w=(None, PTR), dw=(None, PTR)) == OK
    assert go(x=(None, None), w=(None, None), xs=(0, 0), dw=(None, None)) == OK
    assert go(dw=(None, PTR)) == INVALID and go(dw=(PTR, PTR + 4)) == INVALID
    assert go(xs=(6136, 1024)) == INVALID and go(xs=(6144, 1020)) == INVALID
    assert go(ws=PTR + 128) == INVALID and go(ws_bytes=need - 1) == WORKSPACE


@pytest.mark.parametrize("sparse", [False, True])
def test_attn_bwd_refusals(lib, sparse):
    size = lib.msa_sparse_bwd_workspace_bytes if sparse else lib.msa_dense_bwd_workspace_bytes
    fn = lib.msa_sparse_attn_bwd if sparse else lib.msa_dense_attn_bwd
    n_in = 7 if sparse else 6
    need = size(ctypes.byref(P()))
    assert need > 0 and size(ctypes.byref(P(G=9, H=9))) == 0
    assert size(ctypes.byref(P(T=2000))) >= size(ctypes.byref(P(T=100)))

    def go(p=None, ins=None, pos=((0, 0), (0, 0)), outs=(PTR,) * 3, ws=PTR, ws_bytes=need, no_p=False):
        p = p or P()
        ins = [PTR] * n_in if ins is None else ins
        pos = [None if x is None else i32(*x) for x in pos]
        return fn(None if no_p else ctypes.byref(p), *ins, *pos, *outs, ws, ws_bytes, None)
    assert go() == OK and go(no_p=True) == INVALID
    for i in range(n_in):
        for bad in (None, PTR + 4):
            assert go(ins=[PTR] * i + [bad] + [PTR] * (n_in - 1 - i)) == INVALID
    for i in range(3):
        for bad in (None, PTR + 8):
            assert go(outs=[PTR] * i + [bad] + [PTR] * (2 - i)) == INVALID
    assert go(pos=(None, (0, 0))) == INVALID and go(pos=((0, 0), None)) == INVALID
    assert go(p=P(T=5), pos=((0, 0), (5, 4)), ws_bytes=BIG) == INVALID
    assert go(p=P(T=5), pos=((2044, 0), (2049, 5)), ws_bytes=BIG) == INVALID
    assert go(p=P(B=300)) == UNSUPPORTED and go(p=P(scale=float("inf"))) == INVALID
    assert go(ws=None) == INVALID and go(ws=PTR + 16) == INVALID and go(ws_bytes=need - 1) == WORKSPACE


def test_lse_refusals(lib):
    p = P()
    pos = (i32(0, 0), i32(0, 0))
    for lse, want in [(PTR, OK), (None, INVALID), (PTR + 4, INVALID)]:
        assert lib.msa_dense_attn_lse(ctypes.byref(p), PTR, PTR, PTR, *pos, PTR, lse, PTR, BIG,
                                      None) == want
        assert lib.msa_sparse_attn_lse(ctypes.byref(p), PTR, PTR, PTR, PTR, *pos, PTR, lse, PTR, BIG,
                                       None) == want


def test_row_strides():
    p = msa.params(2, 3, 4, 2, 64, 32, 1)
    x = torch.empty(2, 3, 8, 64, dtype=torch.bfloat16)
    q, k, v = x.split([4, 2, 2], 2)
    assert [msa._row_stride(t, p, h, "t") for t, h in ((q, 4), (k, 2), (v, 2))] == [512] * 3
    assert msa._row_stride(x[:, :, :4].contiguous(), p, 4, "q") == 256
    assert msa._row_stride(torch.empty(2, 3, 256), p, 4, "q") == 256
    assert msa._row_stride(12345, p, 4, "q") == 256 and msa._row_stride(None, p, 4, "q") == 256
    for bad in (x, q.transpose(0, 1), q.transpose(2, 3).contiguous().transpose(2, 3), x[:, :, ::2],
                torch.empty(2, 6, 4, 64)[:, :3], q[..., :32]):
        with pytest.raises(ValueError):
            msa._row_stride(bad, p, 4, "q")
    one = msa.params(2, 1, 4, 2, 64, 32, 1)              # a single token: sequences are the rows
    assert msa._row_stride(torch.empty(2, 5, 8, 64)[:, :1, :4], one, 4, "q") == 5 * 512
    one = msa.params(1, 1, 4, 2, 64, 32, 1)
    assert msa._row_stride(torch.empty(1, 1, 8, 64)[:, :, :4], one, 4, "q") == 256


def test_rope_of_bad_sizes():
    for rot in (-2, 3, 130):
        with pytest.raises(ValueError):
            msa.rope(rot)
