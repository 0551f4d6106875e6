"""msa_dense_attn_bwd, msa_sparse_attn_bwd and the forward calls that return lse,
against plain 64-bit forms; the bounds are derived in tests/train_ref.py."""
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
    def __init__(self, B, T, H, G, D, starts, sparse, more=0, extra=1, scale=None, seed=0, size=2.0,
                 skew=0.3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.T, self.H, self.G, self.D = B, T, H, G, D
        self.starts = starts
        self.kv_len = [s + T + more for s in starts]
        self.mb = (max(self.kv_len) + 127) // 128 + extra
        self.scale = D ** -0.5 if scale is None else scale
        self.q, self.dout = bf(g, B, T, H, D, scale=size), bf(g, B, T, H, D)
        self.k, self.v = bf(g, B, self.mb, 128, G, D), bf(g, B, self.mb, 128, G, D)
        j = torch.arange(self.mb * 128, device="cuda")
        self.unseen = j >= torch.tensor(starts, device="cuda")[:, None] + T
        self.behind = j >= torch.tensor(self.kv_len, device="cuda")[:, None]
        self.sel = R.random_sel(T, G, starts, g, "cuda", skew) if sparse else None
        # rows that no query sees hold anything
        for x in (self.k, self.v):
            x.view(B, -1, G, D)[self.unseen] = NAN

    def params(self, msa):
        return msa.params(self.B, self.T, self.H, self.G, self.D, 64, self.mb, scale=self.scale)

    def clean(self, x):
        return torch.where(self.unseen[..., None, None], 0, x.view(self.B, -1, self.G, self.D)).view(
            x.shape)

    def forward_ref(self):
        self.out, self.lse = R.attn_forward(self.q, self.clean(self.k), self.clean(self.v),
                                            self.starts, self.scale, self.sel)

    def backward(self, msa, ws=None, stream=None):
        p = self.params(msa)
        if ws is None:
            ws = msa.dense_bwd_workspace(p) if self.sel is None else msa.sparse_bwd_workspace(p)
            ws.fill_(0xFF)
        self.dq = torch.full_like(self.q, NAN)
        self.dk, self.dv = torch.full_like(self.k, NAN), torch.full_like(self.v, NAN)
        head = (p, self.q, self.k, self.v) + (() if self.sel is None else (self.sel,))
        fn = msa.msa_dense_attn_bwd if self.sel is None else msa.msa_sparse_attn_bwd
        fn(*head, self.out, self.lse, self.dout, self.starts, self.kv_len, self.dq, self.dk, self.dv,
           ws, stream=stream)
        return ws

    def verify(self):
        want, bound = R.attn_backward(self.q, self.clean(self.k), self.clean(self.v), self.out,
                                      self.dout, self.starts, self.kv_len, self.scale, self.sel)
        R.check(self.dq, want[0], bound[0], "dq")
        for got, w, e, what in ((self.dk, want[1], bound[1], "dk"), (self.dv, want[2], bound[2], "dv")):
            flat = got.view(self.B, -1, self.G, self.D)
            assert torch.isnan(flat[self.behind].float()).all(), what + " behind kv_len changed"
            R.check(flat[~self.behind], w.flatten(1, 2)[~self.behind], e.flatten(1, 2)[~self.behind],
                    what)


SHAPES = [
    dict(B=1, T=1, H=4, G=1, D=64, starts=[0]),
    dict(B=1, T=1, H=48, G=8, D=128, starts=[700]),
    dict(B=2, T=2, H=6, G=1, D=128, starts=[0, 127]),
    dict(B=1, T=128, H=4, G=1, D=64, starts=[0]),
    dict(B=1, T=77, H=48, G=8, D=128, starts=[0]),
    dict(B=3, T=130, H=10, G=2, D=64, starts=[0, 51, 300]),
    dict(B=2, T=301, H=64, G=4, D=64, starts=[0, 613], more=40),
    dict(B=2, T=257, H=16, G=1, D=128, starts=[129, 5], more=200),
    dict(B=1, T=700, H=12, G=4, D=128, starts=[0]),
    dict(B=1, T=450, H=7, G=7, D=64, starts=[2000], extra=0),
    dict(B=5, T=33, H=16, G=8, D=128, starts=[0, 1, 127, 128, 1300]),
]


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("kw", SHAPES)
def test_backward(msa, kw, sparse):
    c = Case(sparse=sparse, **kw)
    c.forward_ref()
    ws = c.backward(msa)
    msa.msa_workspace_status(ws)
    c.verify()


@pytest.mark.parametrize("hpg", range(1, 17))
@pytest.mark.parametrize("sparse", [False, True])
def test_heads_per_group(msa, hpg, sparse):
    c = Case(B=1, T=140, H=2 * hpg, G=2, D=64 if hpg % 2 else 128, starts=[250], sparse=sparse, seed=hpg)
    c.forward_ref()
    c.backward(msa)
    c.verify()


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("scale,size", [(-0.1, 2.0), (0.5, 2.0), (0.0, 1.0), (0.125, 0.01)])
def test_scales(msa, sparse, scale, size):
    c = Case(B=1, T=200, H=6, G=1, D=128, starts=[300], sparse=sparse, scale=scale, size=size)
    c.forward_ref()
    c.backward(msa)
    c.verify()


def test_long_context(msa):
    for sparse in (False, True):
        c = Case(B=1, T=70, H=4, G=1, D=64, starts=[30000], sparse=sparse)
        c.forward_ref()
        c.backward(msa)
        c.verify()


def test_many_rows_of_one_block(msa):
    """Nearly every query selects the same blocks: one list holds most of the work."""
    c = Case(B=1, T=2600, H=4, G=1, D=64, starts=[0], sparse=True, skew=50.0)
    c.forward_ref()
    c.backward(msa)
    c.verify()


def test_odd_selections(msa):
    """Ids twice, none at all, out of range, in any order, the local block missing."""
    c = Case(B=1, T=60, H=12, G=2, D=128, starts=[1000], sparse=True)
    s = c.sel
    s[0, 3, 0] = torch.tensor([2, 2, 1] + [-1] * 13, device="cuda")
    s[0, 4] = -1
    s[0, 5, 1] = 0
    s[0, 6, 0] = s[0, 6, 0].flip(0)
    s[0, 7, 1, :] = torch.tensor([-1, 3, -1, 1] + [-1] * 12, device="cuda")
    c.forward_ref()
    ws = c.backward(msa)
    msa.msa_workspace_status(ws)
    c.verify()
    assert (c.dq[0, 4] == 0).all()
    s[0, 8, 0, 2] = 99           # past the local block: reported, skipped
    s[0, 9, 1, 0] = 2 ** 31 - 1
    c.forward_ref()
    ws = c.backward(msa)
    with pytest.raises(msa.MsaError):
        msa.msa_workspace_status(ws)
    c.verify()


def test_no_selection_at_all(msa):
    c = Case(B=2, T=40, H=4, G=2, D=64, starts=[0, 200], sparse=True)
    c.sel.fill_(-1)
    c.out, c.lse = torch.zeros_like(c.q), torch.full((2, 40, 4), -torch.inf, device="cuda")
    c.backward(msa)
    c.verify()
    assert (c.dq == 0).all()


def test_repeats_bit_for_bit(msa):
    for sparse in (False, True):
        c = Case(B=2, T=500, H=12, G=2, D=128, starts=[0, 900], sparse=sparse)
        c.forward_ref()
        c.backward(msa)
        first = [torch.nan_to_num(x) for x in (c.dq, c.dk, c.dv)]
        for _ in range(4):
            c.backward(msa)
            assert all(torch.equal(a, torch.nan_to_num(b)) for a, b in
                       zip(first, (c.dq, c.dk, c.dv)))


@pytest.mark.parametrize("kernels", ["auto", "streaming", "tensorcore"])
@pytest.mark.parametrize("kw", [
    dict(B=2, T=3, H=12, G=2, D=128, starts=[5, 2300]),
    dict(B=1, T=300, H=48, G=8, D=128, starts=[100]),
    dict(B=2, T=70, H=10, G=2, D=64, starts=[0, 2100]),
    dict(B=1, T=9, H=16, G=1, D=64, starts=[0])])
@pytest.mark.parametrize("sparse", [False, True])
def test_forward_lse(msa, kw, sparse, kernels):
    """out has the bits of the call without lse.  lse: scores within (D + 8) 2^-23 S,
    exponentials within 2^-13 (a polynomial in a part of them), sums of positive terms
    in fp32 over N tokens."""
    c = Case(sparse=sparse, size=1.0, **kw)
    c.k, c.v = c.clean(c.k), c.clean(c.v)
    c.forward_ref()
    p = c.params(msa)
    p.kernels = msa.KERNELS[kernels]
    ws = msa.workspace(p) if sparse else msa.dense_workspace(p)
    out, out2 = torch.full_like(c.q, NAN), torch.full_like(c.q, NAN)
    lse = torch.full((c.B, c.T, c.H), NAN, device="cuda")
    if sparse:
        msa.msa_sparse_attn_lse(p, c.q, c.k, c.v, c.sel, c.starts, c.kv_len, out, lse, ws)
        msa.msa_sparse_attn(p, c.q, c.k, c.v, c.sel, c.starts, c.kv_len, out2, ws)
    else:
        msa.msa_dense_attn_lse(p, c.q, c.k, c.v, c.starts, c.kv_len, out, lse, ws)
        msa.msa_dense_attn(p, c.q, c.k, c.v, c.starts, c.kv_len, out2, ws)
    msa.msa_workspace_status(ws)
    assert torch.equal(out, out2)
    S = c.scale * (c.q.double().abs().sum(-1).max() * c.k.double().abs().max())
    N = max(c.starts) + c.T
    bound = (c.D + 8) * 2.0 ** -23 * S + 2.0 ** -13 + (N + 16) * 2.0 ** -23 + 2.0 ** -22 * c.lse.abs()
    R.check(lse, c.lse.double(), bound.double().expand_as(lse), "lse")


def test_forward_lse_of_an_empty_row(msa):
    for kernels in ("streaming", "tensorcore"):
        c = Case(B=1, T=5, H=4, G=2, D=64, starts=[300], sparse=True)
        c.k, c.v = c.clean(c.k), c.clean(c.v)
        c.sel[0, 2, 1] = -1
        p = c.params(msa)
        p.kernels = msa.KERNELS[kernels]
        out, lse = torch.empty_like(c.q), torch.full((1, 5, 4), NAN, device="cuda")
        msa.msa_sparse_attn_lse(p, c.q, c.k, c.v, c.sel, c.starts, c.kv_len, out, lse, msa.workspace(p))
        empty = lse == -torch.inf
        assert empty[0, 2, 2:].all() and empty.sum() == 2 and torch.isfinite(lse[~empty]).all()


@pytest.mark.parametrize("sparse", [False, True])
def test_from_the_library_forward(msa, sparse):
    """Norm and rotation, cache write, forward, backward, backward of the rotation, as a
    layer's training step runs them; the attention's gradients against the 64-bit form
    at the step's own q, caches and out."""
    B, T, H, G, D = 2, 400, 12, 4, 128
    c = Case(B=B, T=T, H=H, G=G, D=D, starts=[0, 200], sparse=sparse)
    g = torch.Generator(device="cuda").manual_seed(9)
    x = bf(g, B, T, H + 2 * G, D)
    q, k, v = x.split([H, G, G], 2)
    qw, kw = 1 + bf(g, D, scale=0.1), 1 + bf(g, D, scale=0.1)
    p = c.params(msa)
    r = msa.rope(64)
    c.k, c.v = c.clean(c.k), c.clean(c.v)         # the second sequence's first 200 tokens
    ws = msa.workspace(p) if sparse else msa.dense_workspace(p)
    msa.msa_rope_append(p, r, q, k, v, None, qw, kw, c.starts, c.q, c.k, c.v, None, ws)
    msa.msa_workspace_status(ws)
    c.out, c.lse = torch.empty_like(c.q), torch.empty(B, T, H, device="cuda")
    if sparse:
        msa.msa_sparse_attn_lse(p, c.q, c.k, c.v, c.sel, c.starts, c.kv_len, c.out, c.lse, ws)
    else:
        msa.msa_dense_attn_lse(p, c.q, c.k, c.v, c.starts, c.kv_len, c.out, c.lse, ws)
    msa.msa_workspace_status(ws)
    bws = c.backward(msa)
    msa.msa_workspace_status(bws)
    c.verify()
    dx = torch.empty_like(x)
    dqw, dkw = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    rws = msa.rope_append_bwd_workspace(p)
    msa.msa_rope_append_bwd(p, r, q, k, qw, kw, c.starts, c.dq, c.dk, c.dv, *dx.split([H, G, G], 2),
                            dqw, dkw, rws)
    msa.msa_workspace_status(rws)
    t = torch.tensor(c.starts, device="cuda")[:, None] + torch.arange(T, device="cuda")
    args = (t, list(r.inv_freq)[:32], False, 1.0, 1e-6)
    rows = [y.view(B, -1, G, D)[torch.arange(B, device="cuda")[:, None], t] for y in (c.dk, c.dv)]
    want, bound, ww, bw = R.norm_rope_bwd(q, qw, c.dq, *args)
    R.check(dx[:, :, :H], want, bound, "projection dq")
    R.check(dqw, ww, bw, "dq_weight")
    want, bound, ww, bw = R.norm_rope_bwd(k, kw, rows[0], *args)
    R.check(dx[:, :, H:H + G], want, bound, "projection dk")
    R.check(dkw, ww, bw, "dk_weight")
    assert torch.equal(dx[:, :, H + G:], rows[1])


def test_graph_and_streams(msa):
    """Captured and replayed on new inputs; two calls at once on two streams."""
    for sparse in (False, True):
        c = Case(B=1, T=200, H=12, G=2, D=128, starts=[150], sparse=sparse)
        c.forward_ref()
        ws = c.backward(msa)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        p = c.params(msa)
        head = (p, c.q, c.k, c.v) + (() if c.sel is None else (c.sel,))
        fn = msa.msa_dense_attn_bwd if c.sel is None else msa.msa_sparse_attn_bwd
        with torch.cuda.graph(graph):
            fn(*head, c.out, c.lse, c.dout, c.starts, c.kv_len, c.dq, c.dk, c.dv, ws)
        for seed in (3, 4):
            g = torch.Generator(device="cuda").manual_seed(seed)
            c.q.copy_(bf(g, *c.q.shape))
            c.dout.copy_(bf(g, *c.dout.shape))
            if sparse:
                c.sel.copy_(R.random_sel(c.T, c.G, c.starts, g, "cuda"))
            out, lse = R.attn_forward(c.q, c.clean(c.k), c.clean(c.v), c.starts, c.scale, c.sel)
            c.out.copy_(out)
            c.lse.copy_(lse)
            graph.replay()
            torch.cuda.synchronize()
            msa.msa_workspace_status(ws)
            c.verify()
    cases = [Case(B=1, T=300 + 7 * i, H=12, G=2, D=64, starts=[i], sparse=i % 2 == 1, seed=i)
             for i in range(4)]
    streams = [torch.cuda.Stream() for _ in cases]
    for c in cases:
        c.forward_ref()
    torch.cuda.synchronize()
    for _ in range(3):
        for c, st in zip(cases, streams):
            with torch.cuda.stream(st):
                c.keep = c.backward(msa)
    torch.cuda.synchronize()
    for c in cases:
        c.verify()


def test_reach_of_a_nan_is_bounded(msa):
    """A NaN in dout of one head reaches that query's dq of that head and dk, dv of its
    group; other groups, and tokens before the tile and behind, keep their gradients."""
    for sparse in (False, True):
        c = Case(B=2, T=300, H=6, G=2, D=64, starts=[0, 300], sparse=sparse)
        c.forward_ref()
        c.dout[1, 100, 4, 3] = NAN
        c.backward(msa)
        bad = ~torch.isfinite(c.dq.float()).all(-1)
        assert bad[1, 100, 4] and bad.sum() == 1
        dk = c.dk.view(2, -1, 2, 64)[1]
        assert torch.isfinite(dk[:600, 0].float()).all()
        assert torch.isfinite(c.dk.view(2, -1, 2, 64)[0, :300].float()).all()
        assert torch.isfinite(dk[512:600, 1].float()).all()


@pytest.mark.parametrize("kw", [
    dict(B=3, T=2790, H=4, G=1, D=64, starts=[0, 500, 77]),
    dict(B=9, T=950, H=3, G=1, D=128, starts=[0, 1, 100, 127, 128, 129, 300, 400, 500])])
def test_more_rows_than_one_pass(msa, kw):
    """Sparse calls of more than 8192 query rows go in passes, which add up dK and dV."""
    c = Case(sparse=True, **kw)
    c.forward_ref()
    ws = c.backward(msa)
    msa.msa_workspace_status(ws)
    c.verify()


def test_offsets_beyond_32_bits(msa):
    """The second sequence's caches begin 2.1e9 elements in: the bits of a small cache."""
    G, D, mb = 8, 128, 16500
    for sparse in (False, True):
        c = Case(B=2, T=40, H=16, G=G, D=D, starts=[3, 300], sparse=sparse)
        c.forward_ref()
        c.backward(msa)
        want = [c.dq, c.dk, c.dv]
        small = c.mb
        c.k, c.v = ([x, torch.empty(2, mb, 128, G, D, dtype=torch.bfloat16, device="cuda")]
                    for x in (c.k, c.v))
        for x in (c.k, c.v):
            x[1][:, :small] = x[0]
        c.k, c.v, c.mb = c.k[1], c.v[1], mb
        p = c.params(msa)
        ws = msa.sparse_bwd_workspace(p) if sparse else msa.dense_bwd_workspace(p)
        dq, dk, dv = torch.empty_like(c.q), torch.empty_like(c.k), torch.empty_like(c.v)
        dk[:, :small], dv[:, :small] = NAN, NAN
        head = (p, c.q, c.k, c.v) + ((c.sel,) if sparse else ())
        fn = msa.msa_sparse_attn_bwd if sparse else msa.msa_dense_attn_bwd
        fn(*head, c.out, c.lse, c.dout, c.starts, c.kv_len, dq, dk, dv, ws)
        msa.msa_workspace_status(ws)
        for got, x in zip((dq, dk[:, :small], dv[:, :small]), want):
            assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(x))
        del dk, dv
        c.k = c.v = None


def test_two_graphs_on_one_workspace(msa):
    """Replayed in turn, each finds the workspace as the other left it."""
    cases = [Case(B=1, T=150, H=12, G=2, D=128, starts=[70], sparse=s, seed=5) for s in (False, True)]
    cases.append(Case(B=2, T=90, H=4, G=1, D=64, starts=[0, 400], sparse=True, seed=6))
    sizes = []
    for c in cases:
        c.forward_ref()
        sizes.append(c.backward(msa).numel())
    ws = torch.empty(max(sizes), dtype=torch.uint8, device="cuda").fill_(0xFF)
    graphs = []
    torch.cuda.synchronize()
    for c in cases:
        p = c.params(msa)
        head = (p, c.q, c.k, c.v) + (() if c.sel is None else (c.sel,))
        fn = msa.msa_dense_attn_bwd if c.sel is None else msa.msa_sparse_attn_bwd
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            fn(*head, c.out, c.lse, c.dout, c.starts, c.kv_len, c.dq, c.dk, c.dv, ws)
    for order in ((0, 1, 2), (2, 1, 0), (1, 1, 0)):
        for c in cases:
            c.dq.fill_(NAN)
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in set(order):
            cases[i].verify()


@pytest.mark.parametrize("sparse,D", [(False, 128), (False, 64), (True, 128), (True, 64)])
def test_wait_expiry_is_reported_then_next_call_is_exact(msa, sparse, D):
    """With a cap of one poll (as in tests/test_gpu_wait_expiry.py) the waits between the
    warps run out on copies that land a moment later: the call reports it, ends, and
    leaves the context and the workspace usable.  Dense, the K and V of a CTA's next unit
    wait for all of its tiles, tens of microseconds; sparse, the same warp copies the tiles'
    rows, so that no wait is longer than two tiles (5 us), which one poll may outlast."""
    c = Case(B=2, T=2000, H=12, G=2, D=D, starts=[500, 0], sparse=sparse)
    c.forward_ref()
    ws = c.backward(msa)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    seen = []
    try:
        msa.msa_debug_set_wait_polls(1)
        for i in range(4):
            flush.fill_(i)
            c.backward(msa, ws)
            try:
                msa.msa_workspace_status(ws)
                seen.append(0)
            except msa.MsaError as e:
                seen.append(e.status)
    finally:
        msa.msa_debug_set_wait_polls(0)
    torch.cuda.synchronize()
    assert set(seen) <= {0, -5} and (sparse or -5 in seen), seen
    c.backward(msa, ws)
    msa.msa_workspace_status(ws)
    c.verify()


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("kw", [
    dict(B=256, T=1, H=16, G=8, D=64, starts=[(61 * i) % 700 for i in range(256)]),
    dict(B=2, T=150, H=128, G=8, D=128, starts=[0, 77])])
def test_most_sequences_and_heads(msa, kw, sparse):
    c = Case(sparse=sparse, **kw)
    c.forward_ref()
    ws = c.backward(msa)
    msa.msa_workspace_status(ws)
    c.verify()
