"""Host-side checks of the serving entry points (8-bit caches, window attention,
page operations): every refusal happens before any CUDA call, so these run
without a GPU on pointers that are never read.  T == 0 and n == 0 are no-ops."""
import ctypes

import pytest

import block_sparse_attention_04_gb300 as msa
from block_sparse_attention_04_gb300 import _build

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
PTR = 0x10000           # 256-byte aligned, never dereferenced
BIG = 1 << 40


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


ATTENTION = {
    # name: (pointer arguments between the pool and the positions, after them)
    "msa_sparse_attn_q8": (6, 1), "msa_forward_q8": (7, 2), "msa_window_attn": (3, 1),
    "msa_window_attn_q8": (5, 1),
}


def call(lib, name, p, table=None, pool=0, ptrs=None, tail=None, q_start=(0, 0), kv_len=(5, 5),
         ws=PTR, ws_bytes=BIG, window=(10, 0)):
    n, m = ATTENTION[name]
    ptrs = [PTR] * n if ptrs is None else ptrs
    tail = [PTR] * m if tail is None else tail
    extra = list(window) if "window" in name else []
    qs = None if q_start is None else i32(*q_start)
    kl = None if kv_len is None else i32(*kv_len)
    return getattr(lib, name)(ctypes.byref(p) if p else None, table, pool, *extra, *ptrs, qs, kl,
                              *tail, ws, ws_bytes, None)


@pytest.mark.parametrize("name", sorted(ATTENTION))
def test_attention_refusals(lib, name):
    n, m = ATTENTION[name]
    assert call(lib, name, P()) == OK
    assert call(lib, name, P(), table=PTR, pool=9) == OK
    assert call(lib, name, None) == INVALID
    assert call(lib, name, P(D=96)) == UNSUPPORTED
    assert call(lib, name, P(G=7)) == INVALID
    assert call(lib, name, P(), table=PTR, pool=0) == INVALID
    assert call(lib, name, P(), table=PTR + 2, pool=9) == INVALID
    assert call(lib, name, P(), table=PTR, pool=1 << 24) == UNSUPPORTED
    for i in range(n):
        for v in (None, PTR + 8):
            bad = [PTR] * n
            bad[i] = v
            assert call(lib, name, P(), ptrs=bad) == INVALID, (i, v)
    for i in range(m):
        for v in (None, PTR + 8):
            bad = [PTR] * m
            bad[i] = v
            optional = name == "msa_forward_q8" and i == 0 and v is None     # sel_out
            assert call(lib, name, P(), tail=bad) == (OK if optional else INVALID)
    assert call(lib, name, P(), q_start=None) == INVALID
    assert call(lib, name, P(), kv_len=None) == INVALID
    assert call(lib, name, P(), q_start=(0, -1)) == INVALID
    assert call(lib, name, P(T=3), kv_len=(3, 2)) == INVALID
    assert call(lib, name, P(), kv_len=(5, 16 * 128 + 1)) == INVALID
    assert call(lib, name, P(), ws=None) == INVALID
    assert call(lib, name, P(), ws=PTR + 128) == INVALID
    size = lib.msa_q8_workspace_bytes if name.endswith("q8") and "window" not in name \
        else lib.msa_window_workspace_bytes
    need = size(ctypes.byref(P()))
    assert need > 0
    assert call(lib, name, P(), ws_bytes=need - 1) == WORKSPACE
    assert call(lib, name, P(), ws_bytes=need) == OK


@pytest.mark.parametrize("name", ["msa_window_attn", "msa_window_attn_q8"])
def test_window_arguments(lib, name):
    for window, sinks, want in [(0, 0, INVALID), (-1, 0, INVALID), (1, -1, INVALID), (1, 0, OK),
                                (2147483647, 2147483647, OK)]:
        assert call(lib, name, P(), window=(window, sinks)) == want


def test_append_q8_refusals(lib):
    def go(p, table=None, pool=0, new=None, cache=None, q_start=(0, 0), ws=PTR, ws_bytes=BIG):
        new = [PTR] * 3 if new is None else new
        cache = [PTR] * 5 if cache is None else cache
        qs = None if q_start is None else i32(*q_start)
        return lib.msa_cache_append_q8(ctypes.byref(p) if p else None, table, pool, *new, qs, *cache,
                                       ws, ws_bytes, None)
    assert go(P()) == OK
    assert go(None) == INVALID
    assert go(P(Di=16)) == UNSUPPORTED
    assert go(P(), table=PTR, pool=-3) == INVALID
    assert go(P(), q_start=None) == INVALID
    assert go(P(T=5), q_start=(0, 16 * 128 - 4)) == INVALID
    assert go(P(), q_start=(-1, 0)) == INVALID
    for i in range(3):
        assert go(P(), new=[PTR] * i + [PTR + 4] + [PTR] * (2 - i)) == INVALID
    for i in range(5):
        assert go(P(), cache=[PTR] * i + [None] + [PTR] * (4 - i)) == INVALID
    assert go(P(), ws=PTR + 16) == INVALID
    assert go(P(), ws_bytes=255) == WORKSPACE


def pool_array(*pools):
    a = (msa.MsaPool * len(pools))()
    for d, (base, size, rows) in zip(a, pools):
        d.base, d.page_bytes, d.per_token = base, size, rows
    return a


POOLS = [(PTR, 128 * 64, 1), (PTR, 8, 0)]


def test_pages_refusals(lib):
    need = lib.msa_pages_workspace_bytes(50)
    assert need > 0 and lib.msa_pages_workspace_bytes(0) == 0
    good = pool_array(*POOLS)

    def copy(pools=good, n_pools=2, pages=50, src=PTR, dst=PTR, n=0, ws=PTR, ws_bytes=need):
        return lib.msa_pages_copy(pools, n_pools, pages, src, dst, n, ws, ws_bytes, None)

    def fork(pools=good, n_pools=2, pages=50, table=PTR, rows=9, mb=4, refs=PTR, src=(), dst=(),
             lens=(), ws=PTR, ws_bytes=need, n=None):
        return lib.msa_pages_fork(pools, n_pools, pages, table, rows, mb, refs, i32(*src), i32(*dst),
                                  i32(*lens), len(src) if n is None else n, ws, ws_bytes, None)

    def ranges(fn, pages=50, table=PTR, rows=9, mb=4, refs=PTR, row=(), first=(), last=(), ws=PTR,
               ws_bytes=need, n=None):
        return fn(pages, table, rows, mb, refs, i32(*row), i32(*first), i32(*last),
                  len(row) if n is None else n, ws, ws_bytes, None)

    def compact(out=(PTR, PTR, PTR), ws_bytes=need, **kw):
        a = dict(pools=good, n_pools=2, pages=50, table=PTR, rows=9, mb=4, refs=PTR)
        a.update(kw)
        return lib.msa_pages_compact(a["pools"], a["n_pools"], a["pages"], a["table"], a["rows"],
                                     a["mb"], a["refs"], *out, PTR, ws_bytes, None)

    assert copy() == fork() == ranges(lib.msa_pages_free) == ranges(lib.msa_pages_alloc) == OK
    for fn in (copy, fork):
        assert fn(n_pools=9) == INVALID and fn(n_pools=-1) == INVALID
        assert fn(pools=None) == INVALID
        assert fn(pools=pool_array((None, 128, 1), POOLS[1])) == INVALID
        assert fn(pools=pool_array((PTR, 0, 1), POOLS[1])) == INVALID
        assert fn(pools=pool_array((PTR, 130, 1), POOLS[1])) == INVALID
        assert fn(pools=pool_array((PTR, 2 << 30, 1), POOLS[1])) == UNSUPPORTED
        assert fn(pages=0) == INVALID
        assert fn(ws=PTR + 1) == INVALID and fn(ws_bytes=need - 1) == WORKSPACE
    assert copy(n=-1) == INVALID and copy(n=1, src=None) == INVALID and copy(src=PTR + 1) == INVALID
    for fn in (fork, lambda **kw: ranges(lib.msa_pages_free, **kw),
               lambda **kw: ranges(lib.msa_pages_alloc, **kw)):
        assert fn(table=None) == INVALID and fn(refs=None) == INVALID
        assert fn(rows=0) == INVALID and fn(mb=0) == INVALID
        assert fn(mb=1 << 24) == UNSUPPORTED and fn(n=-1) == INVALID
        assert fn(n=257) == UNSUPPORTED
        assert fn(ws=None) == INVALID and fn(ws_bytes=0) == WORKSPACE
    for src, dst, lens in [((0,), (9,), (5,)), ((-1,), (1,), (5,)), ((0,), (0,), (5,)),
                           ((0, 1), (2, 2), (5, 5)), ((0, 1), (1, 2), (5, 5)),
                           ((0, 1), (2, 0), (5, 5)), ((0,), (1,), (4 * 128 + 1,)),
                           ((0,), (1,), (-1,))]:
        assert fork(src=src, dst=dst, lens=lens) == INVALID, (src, dst, lens)
    for fn in (lib.msa_pages_free, lib.msa_pages_alloc):
        for r, a, z in [(9, 0, 1), (-1, 0, 1), (0, -1, 1), (0, 2, 1), (0, 0, 5)]:
            assert ranges(fn, row=(r,), first=(a,), last=(z,)) == INVALID
    assert ranges(lib.msa_pages_alloc, row=(1, 1), first=(0, 2), last=(1, 3)) == INVALID
    for i in range(3):
        assert compact(out=[PTR] * i + [None] + [PTR] * (2 - i)) == INVALID
        assert compact(out=[PTR] * i + [PTR + 2] + [PTR] * (2 - i)) == INVALID
    assert compact(table=None) == INVALID and compact(ws_bytes=1) == WORKSPACE


def test_binding_helpers(lib):
    import torch
    a = msa.positions([3, 4])
    assert list(a) == [3, 4] and msa._host_i32(a, 2) is a
    with pytest.raises(ValueError):
        msa._host_i32(a, 3)
    x, y = torch.zeros(6, 128, 2, 64, dtype=torch.uint8), torch.zeros(6, 2, dtype=torch.int8)
    d = msa.pools([x, y])
    assert (d[0].page_bytes, d[0].per_token) == (128 * 128, 1)
    assert (d[1].page_bytes, d[1].per_token) == (2, 0)
    with pytest.raises(ValueError):
        msa.pools([x[:, ::2]])
    lists = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        msa.msa_pages_copy(d, 6, lists, lists[:2], x)
    table = torch.zeros(2, 4, dtype=torch.int32)
    for table_out, refs_out in [(table[:1], lists), (table, lists[:2])]:
        with pytest.raises(ValueError):
            msa.msa_pages_compact(d, 6, table, lists, table_out, refs_out, lists, x)
    assert msa.msa_status_string(-6) == "no free page left"
