"""Page operations (msa_pages_copy, fork, free, alloc, compact) against plain
Python on the host: tables, counts and page contents, exactly."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

PAGES = -6


@pytest.fixture(scope="module")
def msa():
    assert torch.cuda.is_available()
    import block_sparse_attention_04_gb300 as m
    m.load()
    return m


class World:
    """Pools (K-like bf16 rows, 8-bit rows, an odd row size, exponents), a block
    table and counts, on the device and as numpy."""

    def __init__(self, pages, rows, max_blocks, seed, fill=0.5, share=0.0):
        rng = np.random.default_rng(seed)
        self.rng, self.pages = rng, pages
        self.pools = [rng.integers(0, 255, (pages, 128, 2, 64), dtype=np.uint8),
                      rng.integers(0, 1000, (pages, 128, 24)).astype(np.int16),
                      rng.integers(0, 255, (pages, 128, 5), dtype=np.uint8),
                      rng.integers(-99, 99, (pages, 3)).astype(np.int8)]
        self.table = np.full((rows, max_blocks), -1, np.int32)
        self.refs = np.zeros(pages, np.int32)
        perm = list(rng.permutation(pages)[:int(pages * fill)])
        while perm:
            r, kb = rng.integers(rows), rng.integers(max_blocks)
            if self.table[r, kb] < 0:
                self.table[r, kb] = perm.pop()
            if (self.table >= 0).all():
                break
        for r in range(rows):
            for kb in range(max_blocks):
                if rng.random() < share and (self.table >= 0).any():
                    self.table[r, kb] = rng.choice(self.table[self.table >= 0])
        np.add.at(self.refs, self.table[self.table >= 0], 1)

    def device(self, msa):
        self.d_pools = [torch.from_numpy(x.copy()).cuda() for x in self.pools]
        self.d_table = torch.from_numpy(self.table.copy()).cuda()
        self.d_refs = torch.from_numpy(self.refs.copy()).cuda()
        self.set = msa.pools(self.d_pools)
        self.ws = msa.pages_workspace(self.pages)
        self.ws.fill_(0xFF)

    def same(self, table=None, refs=None):
        for got, want in zip(self.d_pools, self.pools):
            assert np.array_equal(got.cpu().numpy(), want)
        table = self.d_table if table is None else table
        refs = self.d_refs if refs is None else refs
        assert np.array_equal(table.cpu().numpy(), self.table)
        assert np.array_equal(refs.cpu().numpy(), self.refs)

    # ---- the plain operations
    def free(self, rows, first, last):
        for r, a, z in zip(rows, first, last):
            for kb in range(a, z):
                if self.table[r, kb] >= 0:
                    self.refs[self.table[r, kb]] -= 1
                self.table[r, kb] = -1

    def take(self):
        ids = np.flatnonzero(self.refs == 0)
        if not len(ids):
            return -1
        self.refs[ids[0]] = 1
        return ids[0]

    def alloc(self, rows, first, last):
        for r, a, z in zip(rows, first, last):
            for kb in range(a, z):
                if self.table[r, kb] == -1:
                    self.table[r, kb] = self.take()

    def fork(self, src, dst, lens):
        for d in dst:
            self.free([d], [0], [self.table.shape[1]])
        for s, d, n in zip(src, dst, lens):
            self.table[d, :n // 128] = self.table[s, :n // 128]
            np.add.at(self.refs, self.table[d, :n // 128], 1)
        for s, d, n in zip(src, dst, lens):
            if n % 128:
                pg = self.take()
                self.table[d, n // 128] = pg
                if pg < 0:
                    continue
                old = self.table[s, n // 128]
                for x in self.pools:
                    if x.ndim > 2:
                        x[pg, :n % 128] = x[old, :n % 128]
                    else:
                        x[pg] = x[old]

    def compact(self):
        live = np.flatnonzero(self.refs > 0)
        n = len(live)
        holes = [i for i in range(n) if self.refs[i] == 0]
        to = np.arange(self.pages)
        for h, m in zip(holes, live[live >= n]):
            to[m] = h
            for x in self.pools:
                x[h] = x[m]
            self.refs[h], self.refs[m] = self.refs[m], 0
        ok = self.table >= 0
        self.table[ok] = to[self.table[ok]]
        return n


def contiguous_world(pages, rows, mb, lens, seed):
    """Rows hold exactly the blocks of `lens` tokens; the rest is unmapped."""
    w = World(pages, rows, mb, seed, fill=0.0)
    perm = iter(w.rng.permutation(pages))
    for r, n in enumerate(lens):
        for kb in range(-(-n // 128)):
            w.table[r, kb] = next(perm)
            w.refs[w.table[r, kb]] = 1
    return w


@pytest.mark.parametrize("seed", range(3))
def test_copy(msa, seed):
    w = World(40, 3, 5, seed)
    ids = w.rng.permutation(40)
    src, dst = ids[:13].astype(np.int32), ids[13:26].astype(np.int32)
    src[4] = src[5]                               # one source twice
    dst[7] = src[7] = ids[30]                     # a pair that does nothing
    w.device(msa)
    msa.msa_pages_copy(w.set, 40, torch.from_numpy(src).cuda(), torch.from_numpy(dst).cuda(), w.ws)
    msa.msa_workspace_status(w.ws)
    for x in w.pools:
        x[dst] = x[src]
    w.same()
    for bad in (-1, 40):
        src[2] = bad
        msa.msa_pages_copy(w.set, 40, torch.from_numpy(src).cuda(), torch.from_numpy(dst).cuda(),
                           w.ws)
        with pytest.raises(msa.MsaError) as e:
            msa.msa_workspace_status(w.ws)
        assert e.value.status == -1
        w.same()


@pytest.mark.parametrize("lens,mb,pages", [
    ([1], 1, 3), ([128, 127, 129], 3, 30), ([1000, 5, 640, 0], 9, 60), ([700] * 40, 6, 1500)])
def test_fork_then_refork_then_free(msa, lens, mb, pages):
    n = len(lens)
    w = contiguous_world(pages, 3 * n, mb, lens, seed=n)
    w.device(msa)
    half = [x // 2 for x in lens]
    steps = [(list(range(n)), list(range(n, 2 * n)), lens),
             ([0] * n, list(range(2 * n, 3 * n)), [lens[0]] * n),
             # rows that are mapped already let go of their pages first
             (list(range(2 * n, 3 * n)), list(range(n, 2 * n)), [min(h, lens[0]) for h in half])]
    for src, dst, ls in steps:
        msa.msa_pages_fork(w.set, pages, w.d_table, w.d_refs, src, dst, ls, w.ws)
        msa.msa_workspace_status(w.ws)
        w.fork(src, dst, ls)
        w.same()
    rows = list(range(3 * n))
    msa.msa_pages_free(pages, w.d_table, w.d_refs, rows, [0] * 3 * n, [mb] * 3 * n, w.ws)
    msa.msa_workspace_status(w.ws)
    assert (w.d_refs == 0).all() and (w.d_table == -1).all()


def test_fork_without_a_free_page(msa):
    w = contiguous_world(7, 6, 3, [300, 300], seed=5)      # 6 pages used, one free
    w.device(msa)
    msa.msa_pages_fork(w.set, 7, w.d_table, w.d_refs, [0, 1, 0], [2, 3, 4], [300, 299, 256], w.ws)
    with pytest.raises(msa.MsaError) as e:
        msa.msa_workspace_status(w.ws)
    assert e.value.status == PAGES
    assert str(e.value) == "kernel status failed: no free page left (-6)"
    w.fork([0, 1, 0], [2, 3, 4], [300, 299, 256])
    assert w.table[3, 2] == -1
    w.same()


@pytest.mark.parametrize("seed", range(4))
def test_free_and_alloc_ranges(msa, seed):
    w = World(3000 if seed == 3 else 200, 8, 11, seed, fill=0.35 if seed < 3 else 0.02, share=0.2)
    w.device(msa)
    rng = w.rng
    for _ in range(4):
        rows = rng.permutation(8)[:5].tolist()
        first = rng.integers(0, 11, 5).tolist()
        last = [int(rng.integers(a, 12)) for a in first]
        rep = rows + rows[:2]                    # a range twice counts once
        msa.msa_pages_free(w.pages, w.d_table, w.d_refs, rep, first + first[:2], last + last[:2],
                           w.ws)
        msa.msa_workspace_status(w.ws)
        w.free(rows, first, last)
        w.same()
        rows = rng.permutation(8)[:4].tolist()
        first, last = [0, 2, 5, 11], [11, 9, 5, 11]
        msa.msa_pages_alloc(w.pages, w.d_table, w.d_refs, rows, first, last, w.ws)
        msa.msa_workspace_status(w.ws)
        w.alloc(rows, first, last)
        w.same()


def test_alloc_runs_out(msa):
    w = World(10, 2, 8, 3, fill=0.3)
    w.device(msa)
    msa.msa_pages_alloc(10, w.d_table, w.d_refs, [1, 0], [0, 0], [8, 8], w.ws)
    with pytest.raises(msa.MsaError) as e:
        msa.msa_workspace_status(w.ws)
    assert e.value.status == PAGES
    w.alloc([1, 0], [0, 0], [8, 8])
    w.same()


@pytest.mark.parametrize("pages,rows,mb,fill,share", [
    (1, 1, 1, 1.0, 0.0), (17, 2, 3, 0.0, 0.0), (64, 8, 8, 1.0, 0.0), (333, 20, 9, 0.4, 0.3),
    (5000, 64, 40, 0.3, 0.05)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(msa, pages, rows, mb, fill, share, in_place):
    w = World(pages, rows, mb, pages, fill=fill, share=share)
    w.device(msa)
    table = w.d_table if in_place else torch.full_like(w.d_table, 77)
    refs = w.d_refs if in_place else torch.full_like(w.d_refs, 77)
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    msa.msa_pages_compact(w.set, pages, w.d_table, w.d_refs, table, refs, live, w.ws)
    msa.msa_workspace_status(w.ws)
    assert live.item() == w.compact()
    w.same(table, refs)
    # compacting again moves nothing
    msa.msa_pages_compact(w.set, pages, table, refs, table, refs, live, w.ws)
    msa.msa_workspace_status(w.ws)
    w.same(table, refs)


def test_sharing_uncounted_pages_is_reported(msa):
    w = contiguous_world(20, 4, 4, [500, 200], seed=19)
    w.device(msa)
    free = [int(i) for i in np.flatnonzero(w.refs == 0)[:2]]
    w.d_table[3, 0], w.d_table[3, 1] = free        # pages whose count stayed 0
    msa.msa_pages_fork(w.set, 20, w.d_table, w.d_refs, [0, 3], [2, 1], [256, 256], w.ws)
    with pytest.raises(msa.MsaError) as e:
        msa.msa_workspace_status(w.ws)
    assert e.value.status == -1
    assert (w.d_refs >= 0).all()
    # the pair beside it is as it should be
    assert np.array_equal(w.d_table[2].cpu().numpy(), list(w.table[0, :2]) + [-1, -1])


def test_inconsistent_tables_are_reported(msa):
    w = contiguous_world(20, 4, 4, [500, 200], seed=9)
    w.device(msa)
    w.d_table[1, 3] = 20                          # outside the pool
    msa.msa_pages_free(20, w.d_table, w.d_refs, [1], [2], [4], w.ws)
    with pytest.raises(msa.MsaError):
        msa.msa_workspace_status(w.ws)
    assert w.d_table[1, 3].item() == -1
    free = int(np.flatnonzero(w.refs == 0)[0])
    w.d_table[1, 3] = free                        # a page that nobody counts
    msa.msa_pages_free(20, w.d_table, w.d_refs, [1], [3], [4], w.ws)
    with pytest.raises(msa.MsaError):
        msa.msa_workspace_status(w.ws)
    assert w.d_refs[free].item() == 0 and (w.d_refs >= 0).all()
    w.d_table[2, 0] = free
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    msa.msa_pages_compact(w.set, 20, w.d_table, w.d_refs, w.d_table, w.d_refs, live, w.ws)
    with pytest.raises(msa.MsaError):
        msa.msa_workspace_status(w.ws)
    # a source row without its pages
    msa.msa_pages_fork(w.set, 20, w.d_table, w.d_refs, [3], [1], [130], w.ws)
    with pytest.raises(msa.MsaError):
        msa.msa_workspace_status(w.ws)
    assert (w.d_table[1] == -1).all()
