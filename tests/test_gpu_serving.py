"""The serving operators together, as a program uses them: prompts appended to
an 8-bit cache through allocated pages, MSA and window attention over it, a
fork with its private last page, decode steps of both branches, freeing the
pages that a window has left, and a compaction; then the same attention calls
captured into CUDA graphs and replayed, on a side stream, and with two graphs
that share a workspace."""
import pytest
import torch

from tests import serving_ref as sr

pytestmark = pytest.mark.gpu

H, G, D, Di, MB = 12, 4, 64, 32, 12
PAGES = 60


@pytest.fixture(scope="module")
def msa():
    assert torch.cuda.is_available()
    import block_sparse_attention_04_gb300 as m
    m.load()
    return m


class Engine:
    """Rows 0 and 1 hold prompts, rows 2 and 3 receive forks."""

    def __init__(self, msa, seed):
        self.msa, self.g = msa, torch.Generator(device="cuda").manual_seed(seed)
        u8 = dict(dtype=torch.uint8, device="cuda")
        self.k = torch.full((PAGES, 128, G, D), 0x7F, **u8)       # NaN until written
        self.v = self.k.clone()
        self.ke = torch.full((PAGES, G), 99, dtype=torch.int8, device="cuda")
        self.ve = self.ke.clone()
        self.ki = torch.zeros(PAGES, 128, Di, dtype=torch.bfloat16, device="cuda")
        self.table = torch.full((4, MB), -1, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(PAGES, dtype=torch.int32, device="cuda")
        self.pools = msa.pools([self.k, self.v, self.ki, self.ke, self.ve])
        self.pws = msa.pages_workspace(PAGES)
        self.aws = torch.empty(256, dtype=torch.uint8, device="cuda")
        self.hist = {}                # row -> (K, V) bf16 values appended so far [n][G][D]

    def ok(self):
        self.msa.msa_workspace_status(self.pws)

    def rand(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda").to(torch.bfloat16)

    def append(self, rows, starts, T):
        B = len(rows)
        first = [s // 128 for s in starts]
        last = [(s + T - 1) // 128 + 1 for s in starts]
        self.msa.msa_pages_alloc(PAGES, self.table, self.refs, rows, first, last, self.pws)
        self.ok()
        kn, vn = self.rand(B, T, G, D), self.rand(B, T, G, D)
        kin = (self.rand(B, T, Di) * 4).round() / 8
        p = self.msa.params(B, T, H, G, D, Di, MB)
        t = self.table[rows].contiguous()
        self.msa.msa_cache_append_q8(p, kn, vn, kin, starts, self.k, self.v, self.ke, self.ve,
                                     self.ki, self.aws, block_table=t, num_pool_blocks=PAGES)
        self.msa.msa_workspace_status(self.aws)
        for i, r in enumerate(rows):
            old = self.hist.get(r)
            new = (kn[i], vn[i])
            self.hist[r] = new if old is None else tuple(torch.cat(x) for x in zip(old, new))

    def values(self, row, n):
        """Cached values of a row's first n tokens, unmapped blocks as zeros."""
        out = []
        for c, e in ((self.k, self.ke), (self.v, self.ve)):
            page = self.table[row].long()
            x = sr.dequant(c[page.clamp(min=0)], e[page.clamp(min=0)])
            x = torch.where((page >= 0)[:, None, None, None], x, 0.0).reshape(-1, G, D)
            out.append(torch.where(torch.arange(x.shape[0], device="cuda")[:, None, None] < n, x, 0))
        return out

    def attend(self, rows, starts, T, window=None, sinks=0, stream=None):
        B, lens = len(rows), [s + T for s in starts]
        q, qi = self.rand(B, T, H, D), (self.rand(B, T, G, Di) * 4).round() / 8
        p = self.msa.params(B, T, H, G, D, Di, MB)
        t = self.table[rows].contiguous()
        out = torch.full_like(q, float("nan"))
        kv = (self.k, self.v, self.ke, self.ve)
        paged = dict(block_table=t, num_pool_blocks=PAGES)
        if window:
            ws = self.msa.window_workspace(p)
            self.msa.msa_window_attn_q8(p, window, sinks, q, *kv, starts, lens, out, ws, **paged)
            seen = sr.window_seen(MB * 128, window, sinks, "cuda")
        else:
            ws = self.msa.q8_workspace(p)
            sel = torch.empty(B, T, G, 16, dtype=torch.int32, device="cuda")
            self.msa.msa_forward_q8(p, qi, self.ki, q, *kv, starts, lens, out, ws, sel_out=sel,
                                    **paged)
        self.msa.msa_workspace_status(ws)
        if not window:
            seen = sr.sel_seen(sel, MB * 128, "cuda")
        k, v = zip(*(self.values(r, n) for r, n in zip(rows, lens)))
        want, bound = sr.attend_call(q, k, v, starts, seen, D ** -0.5, 2 * sr.U_BF16)
        sr.check(out, want, bound)


def test_a_session(msa):
    e = Engine(msa, 1)
    e.append([0, 1], [0, 0], 700)                 # chunk by chunk
    e.append([0, 1], [700, 700], 123)
    e.attend([0, 1], [700, 700], 123)
    e.attend([0, 1], [700, 700], 123, window=300, sinks=4)
    # what is cached is what was appended, within the 8-bit format
    for row in (0, 1):
        for got, want, ex in zip(e.values(row, 823), e.hist[row], (e.ke, e.ve)):
            got, want = got[:823], want.double()
            step = torch.exp2(ex[e.table[row].long().clamp(min=0)].double()).repeat_interleave(128, 0)
            tol = want.abs() * 2.0 ** -4 + step[:823, :, None] * 2.0 ** -9
            assert ((got - want).abs() <= tol).all()
    msa.msa_pages_fork(e.pools, PAGES, e.table, e.refs, [0, 1], [2, 3], [823, 800], e.pws)
    e.ok()
    assert torch.equal(e.table[2, :6], e.table[0, :6])          # complete pages are shared
    assert not torch.equal(e.table[2, 6], e.table[0, 6])
    e.hist[2] = tuple(x.clone() for x in e.hist[0])
    e.hist[3] = tuple(x[:800].clone() for x in e.hist[1])
    pos = [823, 823, 823, 800]
    before = [x.clone() for x in e.values(0, 823)]
    for step in range(3):                         # every branch goes its own way
        e.append([2, 3], pos[2:], 1)
        pos[2], pos[3] = pos[2] + 1, pos[3] + 1
        e.attend([2, 3], [x - 1 for x in pos[2:]], 1)
        e.attend([2, 3], [x - 1 for x in pos[2:]], 1, window=200, sinks=1)
    for a, b in zip(before, e.values(0, 823)):
        assert torch.equal(a, b)
    e.append([0, 1], pos[:2], 1)
    # blocks 1 and 2 have left row 2's window of 300 tokens with one sink block
    e.attend([0, 1, 2, 3], [823, 823, pos[2] - 1, pos[3] - 1], 1, window=300, sinks=128)
    msa.msa_pages_free(PAGES, e.table, e.refs, [2, 3], [1, 1], [3, 3], e.pws)
    e.ok()
    e.attend([2, 3], [pos[2] - 1, pos[3] - 1], 1, window=300, sinks=128)
    msa.msa_pages_free(PAGES, e.table, e.refs, [0], [0], [MB], e.pws)
    e.ok()
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    msa.msa_pages_compact(e.pools, PAGES, e.table, e.refs, e.table, e.refs, live, e.pws)
    e.ok()
    n = live.item()
    assert n == (e.refs > 0).sum().item() and (e.refs[n:] == 0).all()
    e.attend([1], [823], 1)
    e.attend([2, 3], [pos[2] - 1, pos[3] - 1], 1, window=300, sinks=128)


@pytest.mark.parametrize("T", [1, 3, 200])
def test_graphs_that_share_a_workspace(msa, T):
    e = Engine(msa, 2)
    e.append([0, 1], [0, 0], 900)
    lens, starts = [900, 900], [900 - T] * 2
    p = msa.params(2, T, H, G, D, Di, MB)
    q = e.rand(2, T, H, D)
    t = e.table[:2].contiguous()
    kv = (e.k, e.v, e.ke, e.ve)
    paged = dict(block_table=t, num_pool_blocks=PAGES)
    qi = (e.rand(2, T, G, Di) * 4).round() / 8
    n = max(msa.msa_q8_workspace_bytes(p), msa.msa_window_workspace_bytes(p))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def window(out, ws=ws):
        msa.msa_window_attn_q8(p, 333, 5, q, *kv, starts, lens, out, ws, **paged)

    def forward(out, ws=ws):
        msa.msa_forward_q8(p, qi, e.ki, q, *kv, starts, lens, out, ws, **paged)

    def append(out=None):
        msa.msa_cache_append_q8(p, kn, vn, kin, starts, *kv, e.ki, ws, **paged)

    kn, vn, kin = e.rand(2, T, G, D), e.rand(2, T, G, D), e.rand(2, T, Di)
    eager = [torch.empty_like(q) for _ in range(2)]
    append()
    window(eager[0])
    msa.msa_workspace_status(ws)
    forward(eager[1])
    msa.msa_workspace_status(ws)
    torch.cuda.synchronize()
    outs, graphs = [torch.zeros_like(q) for _ in range(2)], []
    side = torch.cuda.Stream()
    for fn, out in zip((window, forward), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            append()
            fn(out)
        graphs.append(g)
    for _ in range(3):
        for g, out, want in zip(graphs, outs, eager):
            out.zero_()
            g.replay()
            msa.msa_workspace_status(ws)
            assert torch.equal(out, want)
    # on another stream, with a workspace of its own, beside the first
    ws2 = torch.empty_like(ws)
    out2 = torch.zeros_like(q)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        window(out2, ws2)
    graphs[1].replay()
    msa.msa_workspace_status(ws2, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out2, eager[0]) and torch.equal(outs[1], eager[1])
    msa.msa_window_attn_q8(p, 333, 5, q, *kv, starts, lens, out2, ws2, stream=side, **paged)
    msa.msa_workspace_status(ws2, stream=side)
    assert torch.equal(out2, eager[0])


def test_pages_in_a_graph(msa):
    e = Engine(msa, 3)
    e.append([0, 1], [0, 0], 300)
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        msa.msa_pages_fork(e.pools, PAGES, e.table, e.refs, [0, 1], [2, 3], [300, 299], e.pws)
        msa.msa_pages_free(PAGES, e.table, e.refs, [2, 3], [0, 0], [1, 1], e.pws)
    want = None
    for _ in range(3):
        g.replay()
        e.ok()
        state = (e.table.clone(), e.refs.clone())
        assert want is None or all(torch.equal(a, b) for a, b in zip(want, state))
        want = state
    assert (e.refs.sum() == (e.table >= 0).sum()).item()
    assert (e.table[2, 0] == -1).item() and (e.refs[e.table[0, 1].long()] == 2).item()
