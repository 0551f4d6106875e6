"""Page operations on tables that map pages which no count owns (count 0, so
free): such mappings are reported and never make two rows share a page unnoticed."""
import numpy as np
import pytest
import torch

from tests.test_gpu_pages import contiguous_world

pytestmark = pytest.mark.gpu

INVALID = -1


@pytest.fixture(scope="module")
def msa():
    assert torch.cuda.is_available()
    import block_sparse_attention_04_gb300 as m
    m.load()
    return m


def reported(msa, ws):
    with pytest.raises(msa.MsaError) as e:
        msa.msa_workspace_status(ws)
    assert e.value.status == INVALID


@pytest.mark.parametrize("which", [0, 1, 2])
def test_fork_does_not_copy_an_uncounted_last_page(msa, which):
    # row 1's last page has count 0 and is the first, second or third free page,
    # i.e. the destination that this pair or another one would get
    w = contiguous_world(30, 8, 4, [300, 290, 257, 0, 500], seed=which + 1)
    free = np.flatnonzero(w.refs == 0)
    w.refs[w.table[1, 2]] = 0
    e = w.table[1, 2] = free[which]
    free = np.flatnonzero(w.refs == 0)
    w.device(msa)
    src, dst, lens = [0, 1, 2], [5, 6, 7], [300, 290, 257]
    msa.msa_pages_fork(w.set, 30, w.d_table, w.d_refs, src, dst, lens, w.ws)
    reported(msa, w.ws)
    for j in (0, 2):                          # the pairs beside it are as they should be
        pg, old, n = free[j], w.table[src[j], 2], lens[j] % 128
        w.table[dst[j], :3] = [*w.table[src[j], :2], pg]
        w.refs[w.table[dst[j], :3]] += 1
        for x in w.pools:
            if x.ndim > 2:
                x[pg, :n] = x[old, :n]
            else:
                x[pg] = x[old]
    w.table[6, :2] = w.table[1, :2]           # complete pages shared, nothing in the last one's place
    w.refs[w.table[6, :2]] += 1
    w.same()
    assert w.table[1, 2] == e and w.refs[e] == int(e in (free[0], free[2]))


def test_fork_copies_a_last_page_that_the_call_itself_shares(msa):
    # the page's own count is there: one pair shares it whole, another copies rows of it
    w = contiguous_world(20, 6, 4, [384, 0, 0], seed=4)
    w.device(msa)
    msa.msa_pages_fork(w.set, 20, w.d_table, w.d_refs, [0, 0], [1, 2], [384, 300], w.ws)
    msa.msa_workspace_status(w.ws)
    w.fork([0, 0], [1, 2], [384, 300])
    w.same()


@pytest.mark.parametrize("in_place", [False, True])
def test_compact_unmaps_uncounted_pages(msa, in_place):
    # entries of a hole that another row's page fills, of a free page behind the
    # live ones, and of no page at all: unmapped, so that every count is the
    # number of entries that map its page
    w = contiguous_world(40, 6, 5, [500, 640, 257], seed=8)
    live = int((w.refs > 0).sum())
    free = np.flatnonzero(w.refs == 0)
    hole, dead = int(free[0]), int(free[-1])
    assert hole < live <= dead
    bad = {(3, 1): hole, (4, 4): dead, (5, 0): 40, (5, 1): -9}
    w.device(msa)
    for at, e in bad.items():
        w.d_table[at] = e
    table = w.d_table if in_place else torch.full_like(w.d_table, 77)
    refs = w.d_refs if in_place else torch.full_like(w.d_refs, 77)
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    msa.msa_pages_compact(w.set, 40, w.d_table, w.d_refs, table, refs, n, w.ws)
    reported(msa, w.ws)
    assert n.item() == w.compact() == live
    w.same(table, refs)                       # the bad entries at -1, the rest as without them
    mapped = table[table >= 0].long()
    assert torch.equal(refs, torch.bincount(mapped, minlength=40).int())


def test_fork_does_not_share_uncounted_pages(msa):
    # two pairs meet the same uncounted page, a third a page of its own kind; the
    # destination rows were mapped before
    w = contiguous_world(40, 9, 4, [500, 384, 130, 300, 200], seed=12)
    a, b = (int(i) for i in np.flatnonzero(w.refs == 0)[:2])
    w.table[0, 1], w.table[2, 0] = a, b       # row 0's block 1 and row 2's block 0: count 0
    w.refs[:] = 0
    np.add.at(w.refs, w.table[w.table >= 0], 1)
    w.refs[[a, b]] = 0
    w.device(msa)
    src, dst, lens = [0, 0, 2, 1], [5, 6, 3, 4], [384, 256, 128, 384]
    msa.msa_pages_fork(w.set, 40, w.d_table, w.d_refs, src, dst, lens, w.ws)
    reported(msa, w.ws)
    w.fork(src, dst, lens)
    w.table[[5, 6, 3], [1, 1, 0]] = -1
    w.refs[[a, b]] = 0
    w.same()
    # every other page is counted once per mapping
    t = w.d_table.clone()
    t[0, 1] = t[2, 0] = -1
    assert torch.equal(w.d_refs, torch.bincount(t[t >= 0].long(), minlength=40).int())
