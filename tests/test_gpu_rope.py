"""msa_rope_append and its backward pass against plain 64-bit forms; the bounds are
derived in tests/train_ref.py."""
import pytest
import torch

from tests import train_ref as R

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module")
def msa():
    assert torch.cuda.is_available()
    import block_sparse_attention_04_gb300 as m
    m.load()
    return m


def bf(gen, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(torch.bfloat16)


class Case:
    """Projections of B x T tokens (parts of one tensor, or three with gaps), caches
    filled with NaN, tables."""

    def __init__(self, B, T, H, G, D, Di, starts, rot, interleaved=False, norm=True, fused=True,
                 paged=False, seed=0, base=10000.0, mscale=1.0, extra=1, index=True):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.T, self.H, self.G, self.D, self.Di = B, T, H, G, D, Di
        self.starts, self.rot, self.interleaved = starts, rot, interleaved
        self.mscale, self.base = mscale, base
        self.mb = (max(starts) + T + 127) // 128 + extra
        if fused:
            self.q, self.k, self.v = bf(g, B, T, H + 2 * G, D, scale=3.0).split([H, G, G], 2)
        else:
            self.q = bf(g, B, T, H * D + 8)[..., :H * D].unflatten(-1, (H, D))
            self.k, self.v = bf(g, B, T, G, D), bf(g, B, T, G + 1, D)[:, :, :G]
        self.qw = 1 + bf(g, D, scale=0.2) if norm else None
        self.kw = 1 + bf(g, D, scale=0.2) if norm else None
        self.ki = bf(g, B, T, Di) if index else None
        pages = B * self.mb + (5 if paged else 0)
        self.pages = pages
        order = torch.randperm(pages, generator=g, device="cuda") if paged else \
            torch.arange(pages, device="cuda")
        self.table = order[:B * self.mb].reshape(B, self.mb).int()
        self.kw_table = dict(block_table=self.table, num_pool_blocks=pages) if paged else {}
        mk = dict(device="cuda", dtype=torch.bfloat16)
        self.kc = torch.full((pages, 128, G, D), NAN, **mk)
        self.vc, self.kic = torch.full_like(self.kc, NAN), torch.full((pages, 128, Di), NAN, **mk)
        self.qo = torch.full((B, T, H, D), NAN, **mk)
        self.t = torch.tensor(starts, device="cuda")[:, None] + torch.arange(T, device="cuda")
        self.page = torch.gather(self.table.long(), 1, self.t // 128)

    def handles(self, msa):
        p = msa.params(self.B, self.T, self.H, self.G, self.D, self.Di, self.mb)
        r = msa.rope(self.rot, base=self.base, interleaved=self.interleaved, mscale=self.mscale)
        return p, r, torch.empty(256, dtype=torch.uint8, device="cuda")

    def freqs(self, r):
        return list(r.inv_freq)[:self.rot // 2]

    def run(self, msa, stream=None):
        p, r, ws = self.handles(msa)
        msa.msa_rope_append(p, r, self.q, self.k, self.v, self.ki, self.qw, self.kw, self.starts,
                            self.qo, self.kc, self.vc, self.kic if self.ki is not None else None, ws,
                            stream=stream, **self.kw_table)
        return ws, r

    def verify(self, r):
        f = self.freqs(r)
        args = (self.t, f, self.interleaved, self.mscale, 1e-6)
        want, bound = R.norm_rope(self.q, self.qw, *args)
        R.check(self.qo, want, bound, "q")
        want, bound = R.norm_rope(self.k, self.kw, *args)
        at = (self.page, self.t % 128)
        R.check(self.kc[at], want, bound, "k")
        assert torch.equal(self.vc[at], self.v)
        written = torch.zeros(self.pages, 128, dtype=torch.bool, device="cuda")
        written[at] = True
        for c in (self.kc, self.vc, self.kic):
            assert torch.isnan(c[~written].float()).all(), "rows that no token owns changed"
        if self.ki is not None:
            assert torch.equal(self.kic[at], self.ki)


CASES = [
    dict(B=1, T=1, H=4, G=1, D=64, Di=32, starts=[0], rot=64),
    dict(B=1, T=1, H=48, G=8, D=128, Di=64, starts=[127], rot=128, paged=True),
    dict(B=64, T=1, H=48, G=8, D=128, Di=64, starts=[(977 * i) % 4096 for i in range(64)], rot=64,
         paged=True),
    dict(B=3, T=77, H=10, G=2, D=64, Di=32, starts=[0, 51, 300], rot=32, interleaved=True, paged=True),
    dict(B=2, T=130, H=64, G=4, D=64, Di=32, starts=[100, 0], rot=48, fused=False),
    dict(B=2, T=65, H=12, G=4, D=128, Di=64, starts=[3, 129], rot=112, interleaved=True, fused=False),
    dict(B=1, T=33, H=7, G=7, D=128, Di=32, starts=[1], rot=0),
    dict(B=1, T=40, H=16, G=1, D=128, Di=64, starts=[10], rot=16, norm=False, index=False),
    dict(B=2, T=3, H=5, G=1, D=64, Di=64, starts=[0, 7], rot=0, norm=False, fused=False),
    dict(B=2, T=3, H=5, G=1, D=64, Di=64, starts=[0, 7], rot=64, mscale=1.37, base=5e6, norm=False),
    dict(B=1, T=3000, H=12, G=4, D=128, Di=64, starts=[90], rot=128, interleaved=True),
]


@pytest.mark.parametrize("kw", CASES)
def test_append(msa, kw):
    c = Case(**kw)
    ws, r = c.run(msa)
    msa.msa_workspace_status(ws)
    c.verify(r)


def test_far_positions(msa):
    """The last positions of the longest context: angles of four million turns."""
    n = 32768 * 128
    c = Case(B=1, T=5, H=4, G=1, D=64, Di=32, starts=[n - 5], rot=64, extra=0)
    ws, r = c.run(msa)
    msa.msa_workspace_status(ws)
    c.verify(r)


def test_yarn_frequencies(msa):
    r = msa.rope(64, base=10000.0, yarn=(16.0, 4096), mscale=msa.yarn_mscale(16.0))
    want = R.yarn_freqs(64, 10000.0, 16.0, 4096)
    assert all(abs(a - b) <= 1e-12 * b for a, b in zip(list(r.inv_freq), want))
    assert want[0] == 1.0 and want[-1] < 10000.0 ** (-62 / 64) / 15
    r = msa.rope(32, linear=4.0)
    assert abs(r.inv_freq[0] - 0.25) < 1e-15


def test_bad_table_entry(msa):
    c = Case(B=2, T=4, H=4, G=2, D=64, Di=32, starts=[10, 200], rot=64, paged=True)
    c.table[1, 1] = c.pages + 3
    ws, r = c.run(msa)
    with pytest.raises(msa.MsaError):
        msa.msa_workspace_status(ws)
    want, bound = R.norm_rope(c.q, c.qw, c.t, c.freqs(r), False, 1.0, 1e-6)
    R.check(c.qo, want, bound, "q")
    at = (c.page[0], c.t[0] % 128)
    assert torch.equal(c.vc[at], c.v[0])
    left = torch.ones(c.pages, 128, dtype=torch.bool, device="cuda")
    left[at] = False
    assert torch.isnan(c.kc[left].float()).all() and torch.isnan(c.kic[left].float()).all()


def test_non_finite_rows_stay_in_their_head(msa):
    c = Case(B=1, T=4, H=4, G=2, D=64, Di=32, starts=[0], rot=64, fused=False)
    c.q[0, 1, 2, 5] = NAN
    c.k[0, 2, 0, 3] = float("inf")
    ws, r = c.run(msa)
    bad = ~torch.isfinite(c.qo.float()).all(-1)[0]
    assert bad.sum() == 1 and bad[1, 2]
    bad = ~torch.isfinite(c.kc[0, :4].float()).all(-1)
    assert bad.sum() == 1 and bad[2, 0]
    # rotation alone: a NaN reaches its pair
    c = Case(B=1, T=4, H=4, G=2, D=64, Di=32, starts=[0], rot=32, norm=False, fused=False)
    c.q[0, 1, 2, 5] = NAN
    c.run(msa)
    assert torch.isnan(c.qo.float()).nonzero().tolist() == [[0, 1, 2, 5], [0, 1, 2, 21]]


def run_bwd(msa, c, stream=None, seed=5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    p, r, _ = c.handles(msa)
    ws = msa.rope_append_bwd_workspace(p)
    c.dqo = bf(g, c.B, c.T, c.H, c.D)
    c.dkc, c.dvc = bf(g, c.B, c.mb, 128, c.G, c.D), bf(g, c.B, c.mb, 128, c.G, c.D)
    own = torch.arange(c.mb * 128, device="cuda")
    own = (own >= c.t[:, :1]) & (own <= c.t[:, -1:])
    for x in (c.dkc, c.dvc):       # gradients of other tokens are not read
        x.view(c.B, -1, c.G, c.D)[~own] = NAN
    mk = dict(device="cuda", dtype=torch.bfloat16)
    c.grads = torch.full((c.B, c.T, c.H + 2 * c.G + 1, c.D), NAN, **mk)
    c.dq, c.dk, c.dv, _ = c.grads.split([c.H, c.G, c.G, 1], 2)
    c.dqw, c.dkw = (torch.full((c.D,), NAN, device="cuda") for _ in range(2))
    msa.msa_rope_append_bwd(p, r, c.q, c.k, c.qw, c.kw, c.starts, c.dqo, c.dkc, c.dvc, c.dq, c.dk,
                            c.dv, c.dqw, c.dkw, ws, stream=stream)
    c.own = own
    return ws, r


def verify_bwd(c, r):
    args = (c.t, c.freqs(r), c.interleaved, c.mscale, 1e-6)

    def rows(x):
        return x.view(c.B, -1, c.G, c.D)[c.own].view(c.B, c.T, c.G, c.D)

    for x, w, dy, dx, dw, what in ((c.q, c.qw, c.dqo, c.dq, c.dqw, "dq"),
                                   (c.k, c.kw, rows(c.dkc), c.dk, c.dkw, "dk")):
        want, bound, want_w, bound_w = R.norm_rope_bwd(x, w, dy, *args)
        R.check(dx, want, bound, what)
        if w is None:
            assert torch.isnan(dw).all()
        else:
            R.check(dw, want_w, bound_w, what + "_weight")
    assert torch.equal(c.dv, rows(c.dvc))
    assert torch.isnan(c.grads[:, :, -1].float()).all()


@pytest.mark.parametrize("kw", [k for k in CASES if not k.get("paged")] + [
    dict(B=3, T=77, H=10, G=2, D=64, Di=32, starts=[0, 51, 300], rot=32, interleaved=True),
    dict(B=5, T=1001, H=48, G=8, D=128, Di=64, starts=[0, 5, 10, 15, 20], rot=96)])
def test_append_backward(msa, kw):
    c = Case(**kw)
    ws, r = run_bwd(msa, c)
    msa.msa_workspace_status(ws)
    verify_bwd(c, r)


def test_one_norm_only(msa):
    """A norm of the queries alone: the keys' projections are not read."""
    c = Case(B=1, T=9, H=4, G=2, D=64, Di=32, starts=[4], rot=64)
    c.kw = None
    ws, r = c.run(msa)
    c.verify(r)
    c.k = None
    p, _, _ = c.handles(msa)
    ws, r = run_bwd(msa, c)
    c.k = torch.zeros(1, 9, 2, 64, device="cuda")
    verify_bwd(c, r)


def test_backward_repeats_bit_for_bit(msa):
    c = Case(B=2, T=777, H=48, G=8, D=128, Di=64, starts=[0, 90], rot=128)
    run_bwd(msa, c)
    first = [x.clone() for x in (c.grads, c.dqw, c.dkw)]
    for _ in range(3):
        run_bwd(msa, c)
        for a, b in zip(first, (c.grads, c.dqw, c.dkw)):
            assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))


def test_graph_and_streams(msa):
    """Captured and replayed on new inputs; two streams at once, each with its own ws."""
    c = Case(B=2, T=70, H=12, G=4, D=128, Di=64, starts=[5, 60], rot=128)
    c.run(msa)
    run_bwd(msa, c)
    torch.cuda.synchronize()
    p, r, ws = c.handles(msa)
    ws2 = msa.rope_append_bwd_workspace(p)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        msa.msa_rope_append(p, r, c.q, c.k, c.v, c.ki, c.qw, c.kw, c.starts, c.qo, c.kc, c.vc, c.kic,
                            ws)
        msa.msa_rope_append_bwd(p, r, c.q, c.k, c.qw, c.kw, c.starts, c.dqo, c.dkc, c.dvc, c.dq,
                                c.dk, c.dv, c.dqw, c.dkw, ws2)
    for seed in (1, 2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        c.q.copy_(bf(g, *c.q.shape))
        c.dqo.copy_(bf(g, *c.dqo.shape))
        graph.replay()
        torch.cuda.synchronize()
        c.verify(r)
        verify_bwd(c, r)
    cases = [Case(B=1, T=400 + i, H=12, G=4, D=64, Di=32, starts=[i], rot=64, seed=i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, st in zip(cases, streams):
            with torch.cuda.stream(st):
                c.keep = c.run(msa)
    torch.cuda.synchronize()
    for c in cases:
        c.verify(c.keep[1])


def test_no_tokens(msa):
    """A call without tokens writes nothing, not the weights' gradients either."""
    p = msa.params(2, 0, 4, 2, 64, 32, 3)
    r = msa.rope(64)
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    cache = [torch.full((2, 3, 128, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    dqw, dkw = torch.full((64,), 3.0, device="cuda"), torch.full((64,), 3.0, device="cuda")
    some = torch.full((64,), 3.0, dtype=torch.bfloat16, device="cuda")
    a = some.data_ptr()      # tensors without elements have no address
    msa.msa_rope_append(p, r, a, a, a, None, w, w, [0, 5], a, *cache, None, msa.workspace(p))
    msa.msa_rope_append_bwd(p, r, a, a, w, w, [0, 5], a, *cache, a, a, a, dqw, dkw,
                            msa.rope_append_bwd_workspace(p))
    torch.cuda.synchronize()
    assert all((x == 3).all() for x in (*cache, dqw, dkw, some))


def test_only_the_entries_of_the_call_count(msa):
    """Table entries that no token of the call falls into may hold anything; one bad entry
    of the last sequence's last block is found."""
    c = Case(B=70, T=130, H=4, G=2, D=64, Di=32, starts=[7 * b for b in range(70)], rot=64, paged=True)
    first = torch.tensor(c.starts, device="cuda") // 128
    last = (torch.tensor(c.starts, device="cuda") + 129) // 128
    kb = torch.arange(c.table.shape[1], device="cuda")
    c.table[(kb < first[:, None]) | (kb > last[:, None])] = -5
    ws, _ = c.run(msa)
    msa.msa_workspace_status(ws)
    c.table[69, last[69]] = 2 ** 31 - 1
    ws, _ = c.run(msa)
    with pytest.raises(msa.MsaError):
        msa.msa_workspace_status(ws)


@pytest.mark.parametrize("kw", [
    dict(B=256, T=1, H=16, G=8, D=64, Di=32, starts=[(61 * i) % 700 for i in range(256)], rot=64),
    dict(B=3, T=70, H=128, G=8, D=128, Di=64, starts=[0, 60, 127], rot=128)])
def test_most_sequences_and_heads(msa, kw):
    c = Case(paged=True, **kw)
    ws, r = c.run(msa)
    msa.msa_workspace_status(ws)
    c.verify(r)
    test_append_backward(msa, kw)
