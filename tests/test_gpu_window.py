"""Sliding-window attention with sinks (msa_window_attn, msa_window_attn_q8)
against 64-bit attention, within the bounds of serving_ref: windows from one
token to past the context, sinks inside and outside the window, odd sizes, both
caches, both kernel families.  Cache rows that no query sees hold NaN, and so
do the table entries of blocks without a visible token."""
import pytest
import torch

from tests import serving_ref as sr
from tests.test_gpu_cache_q8 import Cache

pytestmark = pytest.mark.gpu

KERNELS = ["streaming", "tensorcore", "auto"]


@pytest.fixture(scope="module")
def msa():
    assert torch.cuda.is_available()
    import block_sparse_attention_04_gb300 as m
    m.load()
    return m


def bf16_cache(c):
    """The bf16 cache of a Cache's values (codes become NaN where it holds NaN)."""
    return [sr.dequant(x, e).to(torch.bfloat16) for x, e in zip(c.codes, c.exps)]


def visible_blocks(table, q_start, T, window, sinks):
    """The table with every entry whose block no query of the call sees set to a
    value far outside the pool."""
    out = torch.full_like(table, -(1 << 30))
    for b, a in enumerate(q_start):
        lo = max(0, a - window + 1) // 128
        ns = min(-(-sinks // 128), (a + T - 1) // 128 + 1)
        out[b, :ns] = table[b, :ns]
        out[b, lo:(a + T - 1) // 128 + 1] = table[b, lo:(a + T - 1) // 128 + 1]
    return out


def run(msa, c, q8, q, q_start, kv_len, nb, window, sinks, kernels, scale=None, paged=True,
        kv=None, trim=True):
    B, T, H, D = q.shape
    G = c.codes[0].shape[2]
    p = msa.params(B, T, H, G, D, 32, nb, kernels=kernels, scale=scale)
    ws = msa.window_workspace(p)
    ws.fill_(0xFF)
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    kv = kv or ((*c.codes, *c.exps) if q8 else bf16_cache(c))
    kw = {}
    if paged:
        table = visible_blocks(c.table, q_start, T, window, sinks) if trim else c.table
        kw = dict(block_table=table, num_pool_blocks=c.pages)
    else:
        kv = [x[c.table.long().reshape(-1)].contiguous() for x in kv]
    fn = msa.msa_window_attn_q8 if q8 else msa.msa_window_attn
    fn(p, window, sinks, q, *kv, q_start, kv_len, out, ws, **kw)
    msa.msa_workspace_status(ws)
    return out


def make(lens, T, H, G, D, seed, extra=0, nb=None):
    c = Cache([n + extra for n in lens], G, D, nb or max(-(-(n + extra) // 128) for n in lens) + 1,
              seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = torch.randn(len(lens), T, H, D, generator=g, device="cuda").to(torch.bfloat16)
    return c, q, [n - T for n in lens]


CASES = [
    # lens, T, H, G, D, window, sinks
    ([1, 127, 128, 129, 5000], 1, 48, 8, 128, 1, 0),
    ([1, 2, 300, 2049, 5001], 1, 48, 8, 128, 128, 4),
    ([901, 7], 1, 4, 1, 64, 512, 0),
    ([3000, 1200], 1, 64, 4, 64, 1 << 22, 0),
    ([2000, 640], 1, 16, 1, 128, 129, 300),
    ([1111, 5, 300], 3, 10, 2, 64, 127, 1),
    ([700, 701], 7, 12, 4, 128, 3, 2000),
    ([1500], 517, 12, 4, 128, 200, 5),
    ([777, 1300], 255, 64, 4, 64, 130, 0),
    ([600], 600, 10, 2, 128, 1, 1),
    ([900], 900, 4, 4, 64, 1000, 0),
    ([1025], 640, 6, 2, 64, 129, 128),
    ([2500], 129, 48, 8, 128, 640, 130),
    ([400, 401, 402], 128, 16, 1, 64, 64, 64),
]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kernels", KERNELS)
@pytest.mark.parametrize("lens,T,H,G,D,window,sinks", CASES)
def test_window(msa, lens, T, H, G, D, window, sinks, kernels, q8):
    c, q, q_start = make(lens, T, H, G, D, seed=len(lens) * 100 + T)
    nb = c.table.shape[1]
    out = run(msa, c, q8, q, q_start, lens, nb, window, sinks, kernels)
    k, v = c.values()
    want, bound = sr.attend_call(q, k, v, q_start, sr.window_seen(nb * 128, window, sinks, "cuda"),
                                 D ** -0.5, sr.U_BF16)
    sr.check(out, want, bound)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("T", [1, 9, 50])
def test_split_block_lists(msa, T, q8):
    # few tiles, long lists: the tensor-core kernel splits every list over several
    # items; the short sequence's list is shorter than the number of parts
    lens = [9000, 60, 700]
    c, q, q_start = make(lens, T, 12, 2, 64, seed=74)
    nb = c.table.shape[1]
    out = run(msa, c, q8, q, q_start, lens, nb, 1 << 22, 3, "tensorcore")
    k, v = c.values()
    want, bound = sr.attend_call(q, k, v, q_start, sr.window_seen(nb * 128, 1 << 22, 3, "cuda"),
                                 0.125, sr.U_BF16)
    sr.check(out, want, bound)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("H,G,D", [(48, 8, 128), (24, 8, 64), (64, 4, 128), (8, 8, 128)])
def test_long_decode_laps_every_ring(msa, H, G, D, q8):
    # about 30 blocks per CTA: every stage of the block ring is reused several
    # times, by both teams of warps where there are two
    lens = [18000, 17000, 16500, 11111]
    c, q, q_start = make(lens, 1, H, G, D, seed=73)
    nb = c.table.shape[1]
    out = run(msa, c, q8, q, q_start, lens, nb, 1 << 22, 0, "streaming")
    k, v = c.values()
    want, bound = sr.attend_call(q, k, v, q_start, sr.window_seen(nb * 128, 1 << 22, 0, "cuda"),
                                 D ** -0.5, sr.U_BF16)
    sr.check(out, want, bound)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kernels", KERNELS)
def test_window_past_the_context_is_dense_attention(msa, kernels, q8):
    # kv_len beyond the last query: the tokens behind it are not seen
    c, q, q_start = make([1400, 900], 300, 12, 4, 128, seed=71, extra=200)
    kv_len = [1600, 1100]
    nb = c.table.shape[1]
    out = run(msa, c, q8, q, q_start, kv_len, nb, 1 << 30, 1 << 30, kernels)
    k, v = c.values()
    want, bound = sr.attend_call(q, k, v, q_start, sr.window_seen(nb * 128, 1 << 30, 0, "cuda"),
                                 128 ** -0.5, sr.U_BF16)
    sr.check(out, want, bound)
    if not q8:
        p = msa.params(2, 300, 12, 4, 128, 32, nb, kernels=kernels)
        kv = [torch.nan_to_num(x)[c.table.long().reshape(-1)].contiguous() for x in bf16_cache(c)]
        dense, ws = torch.empty_like(out), msa.dense_workspace(p)
        msa.msa_dense_attn(p, q, *kv, q_start, kv_len, dense, ws)
        msa.msa_workspace_status(ws)
        sr.check(dense, want, bound)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kernels", KERNELS)
@pytest.mark.parametrize("scale", [4.0, -0.3, 0.0])
def test_window_scales(msa, kernels, q8, scale):
    c, q, q_start = make([800, 333], 140, 10, 2, 64, seed=81)
    nb = c.table.shape[1]
    out = run(msa, c, q8, q, q_start, [800, 333], nb, 200, 9, kernels, scale=scale)
    k, v = c.values()
    want, bound = sr.attend_call(q, k, v, q_start, sr.window_seen(nb * 128, 200, 9, "cuda"), scale,
                                 sr.U_BF16)
    sr.check(out, want, bound)


@pytest.mark.parametrize("kernels", KERNELS)
def test_window_q8_spread_exponents(msa, kernels):
    c, q, q_start = make([1300, 800], 130, 16, 2, 64, seed=85)
    nb = c.table.shape[1]
    g = torch.Generator(device="cuda").manual_seed(86)
    c.exps[0] = torch.randint(-50, -8, c.exps[0].shape, generator=g, device="cuda", dtype=torch.int8)
    c.exps[1] = torch.randint(-60, 30, c.exps[1].shape, generator=g, device="cuda", dtype=torch.int8)
    out = run(msa, c, True, q, q_start, [1300, 800], nb, 700, 9, kernels)
    k, v = c.values()
    want, bound = sr.attend_call(q, k, v, q_start, sr.window_seen(nb * 128, 700, 9, "cuda"),
                                 64 ** -0.5, sr.U_BF16)
    sr.check(out, want, bound)


@pytest.mark.parametrize("kernels", KERNELS)
@pytest.mark.parametrize("T", [1, 140])
def test_window_q8_blocks_of_zeros_keep_their_weight(msa, kernels, T):
    c, q, q_start = make([1100], T, 12, 2, 128, seed=87)
    nb = c.table.shape[1]
    for i in (0, 5, 8):
        page = c.table[0, i].long()
        c.codes[1][page] = torch.where(c.codes[1][page] == 0x7F, c.codes[1][page], 0)
        c.exps[1][page] = -126
    c.exps[1][c.table[0, 6].long()] = 60
    loud = c.table[0, 3].long()                 # zeros under a large exponent
    c.codes[1][loud], c.exps[1][loud] = 0, 30
    for scale in (0.01, 0.3):
        out = run(msa, c, True, q, q_start, [1100], nb, 800, 9, kernels, scale=scale)
        k, v = c.values()
        want, bound = sr.attend_call(q, k, v, q_start, sr.window_seen(nb * 128, 800, 9, "cuda"),
                                     scale, sr.U_BF16)
        sr.check(out, want, bound)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kernels", KERNELS)
def test_window_per_sequence_equals_paged(msa, kernels, q8):
    c, q, q_start = make([1000, 640], 33, 12, 4, 128, seed=91)
    nb = c.table.shape[1]
    args = (msa, c, q8, q, q_start, [1000, 640], nb, 300, 7, kernels)
    assert torch.equal(run(*args), run(*args, paged=False))


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kernels", KERNELS)
def test_rows_behind_the_last_sequence_stay(msa, kernels, q8):
    c, q, q_start = make([300, 200], 70, 4, 2, 64, seed=95)
    nb = c.table.shape[1]
    p = msa.params(2, 70, 4, 2, 64, 32, nb, kernels=kernels)
    ws = msa.window_workspace(p)
    out = torch.full((3, 70, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    kv = (*c.codes, *c.exps) if q8 else bf16_cache(c)
    fn = msa.msa_window_attn_q8 if q8 else msa.msa_window_attn
    fn(p, 50, 3, q, *kv, q_start, [300, 200], out, ws, block_table=c.table, num_pool_blocks=c.pages)
    msa.msa_workspace_status(ws)
    assert (out[2] == 7.0).all() and torch.isfinite(out[:2]).all() and (out[:2] != 7.0).any()


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kernels", KERNELS)
def test_window_bad_table_entry_is_reported(msa, kernels, q8):
    c, q, q_start = make([900], 140, 4, 2, 64, seed=97)
    nb = c.table.shape[1]
    p = msa.params(1, 140, 4, 2, 64, 32, nb, kernels=kernels)
    ws = msa.window_workspace(p)
    out = torch.empty_like(q)
    kv = (*c.codes, *c.exps) if q8 else bf16_cache(c)
    table = c.table.clone()
    table[0, 6] = -5
    fn = msa.msa_window_attn_q8 if q8 else msa.msa_window_attn
    fn(p, 1 << 20, 0, q, *kv, q_start, [900], out, ws, block_table=table, num_pool_blocks=c.pages)
    with pytest.raises(msa.MsaError) as e:
        msa.msa_workspace_status(ws)
    assert e.value.status == -1
    fn(p, 1 << 20, 0, q, *kv, q_start, [900], out, ws, block_table=c.table, num_pool_blocks=c.pages)
    msa.msa_workspace_status(ws)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kernels", KERNELS)
def test_nan_in_a_visible_token_is_seen(msa, kernels, q8):
    # one decode step per sequence: a NaN in K of a visible token makes the
    # heads of its group NaN, one in V the dim it sits in; other outputs stay
    c, q, q_start = make([500, 500, 500], 1, 4, 2, 64, seed=99)
    nb = c.table.shape[1]
    pos = 450

    def put(x, b, g, d, val):
        x[c.table[b, pos // 128].long(), pos % 128, g, d] = val
    if q8:
        kv = [x.clone() for x in c.codes]
        put(kv[0], 0, 0, 3, 0x7F)
        put(kv[1], 1, 1, 5, 0xFF)
        kv += c.exps
    else:
        kv = bf16_cache(c)
        put(kv[0], 0, 0, 3, float("nan"))
        put(kv[1], 1, 1, 5, float("nan"))
    out = run(msa, c, q8, q, q_start, [500] * 3, nb, 100, 0, kernels, kv=kv)
    nan = out.isnan()
    want = torch.zeros_like(nan)
    want[0, 0, :2] = True
    want[1, 0, 2:, 5] = True
    assert torch.equal(nan, want)
    # the same tokens outside the window change nothing
    out = run(msa, c, q8, q, q_start, [500] * 3, nb, 40, 5, kernels, kv=kv)
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("kernels", KERNELS)
def test_window_all_scores_minus_infinity_then_finite(msa, kernels):
    # K rows of -inf in one block (scores of -inf for positive queries) take no
    # weight; finite blocks before and after decide the result
    c, q, q_start = make([700], 1, 4, 2, 64, seed=103)
    q = q.abs() + 0.1
    kv = bf16_cache(c)
    page = c.table[0, 2].long()
    kv[0][page] = float("-inf")
    out = run(msa, c, False, q, q_start, [700], c.table.shape[1], 1 << 20, 0, kernels, kv=kv)
    k, v = c.values()
    k[0][256:384] = 0
    base = sr.window_seen(k[0].shape[0], 1 << 20, 0, "cuda")

    def seen(b, g, t):
        s = base(b, g, t).clone()
        s[:, 256:384] = False
        return s
    want, bound = sr.attend_call(q, k, v, q_start, seen, 64 ** -0.5, sr.U_BF16)
    sr.check(out, want, bound)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("H,G", [(12, 3), (5, 5), (18, 6), (14, 7)])
def test_window_any_number_of_kv_heads(msa, H, G, q8):
    # runs of blocks are shared by G CTAs each, whatever G leaves of the SMs
    lens = [6000, 4100, 130]
    c, q, q_start = make(lens, 2, H, G, 64, seed=H)
    nb = c.table.shape[1]
    out = run(msa, c, q8, q, q_start, lens, nb, 5000, 70, "streaming")
    k, v = c.values()
    want, bound = sr.attend_call(q, k, v, q_start, sr.window_seen(nb * 128, 5000, 70, "cuda"),
                                 0.125, sr.U_BF16)
    sr.check(out, want, bound)


@pytest.mark.parametrize("q8", [False, True])
def test_streaming_in_several_passes_joins_their_status(msa, q8):
    # 2 x 1300 queries: more than one pass of the streaming kernels.  A bad entry
    # that only queries of the first pass read is still reported at the end.
    lens, T, window = [1300, 1500], 1300, 100
    c, q, q_start = make(lens, T, 4, 2, 64, seed=41)
    nb = c.table.shape[1]
    out = run(msa, c, q8, q, q_start, lens, nb, window, 0, "streaming")
    k, v = c.values()
    want, bound = sr.attend_call(q, k, v, q_start, sr.window_seen(nb * 128, window, 0, "cuda"),
                                 0.125, sr.U_BF16)
    sr.check(out, want, bound)
    p = msa.params(2, T, 4, 2, 64, 32, nb, kernels="streaming")
    ws = msa.window_workspace(p)
    kv = (*c.codes, *c.exps) if q8 else bf16_cache(c)
    fn = msa.msa_window_attn_q8 if q8 else msa.msa_window_attn
    table = c.table.clone()
    table[0, 1] = c.pages
    got = torch.empty_like(out)
    fn(p, window, 0, q, *kv, q_start, lens, got, ws, block_table=table, num_pool_blocks=c.pages)
    with pytest.raises(msa.MsaError) as e:
        msa.msa_workspace_status(ws)
    assert e.value.status == -1
    assert torch.equal(got[1], out[1]) and torch.equal(got[0, 400:], out[0, 400:])


@pytest.mark.parametrize("kernels", KERNELS)
def test_window_of_the_largest_batch(msa, kernels):
    # 256 sequences, nine tokens each: two streaming passes of eight queries
    lens = [9 + (37 * i) % 400 for i in range(256)]
    c, q, q_start = make(lens, 9, 2, 1, 64, seed=43)
    nb = c.table.shape[1]
    for q8 in (False, True):
        out = run(msa, c, q8, q, q_start, lens, nb, 150, 3, kernels)
        k, v = c.values()
        want, bound = sr.attend_call(q, k, v, q_start, sr.window_seen(nb * 128, 150, 3, "cuda"),
                                     0.125, sr.U_BF16)
        sr.check(out, want, bound)


def test_two_calls_at_once_on_two_streams(msa):
    # the same inputs on two side streams, with a workspace each
    lens = [5000, 3000, 700]
    c, q, q_start = make(lens, 40, 12, 4, 128, seed=47)
    nb = c.table.shape[1]
    calls = []
    for kernels in ("streaming", "tensorcore"):
        p = msa.params(3, 40, 12, 4, 128, 32, nb, kernels=kernels)
        calls.append((p, msa.window_workspace(p), torch.empty_like(q), torch.cuda.Stream()))
    args = ((*c.codes, *c.exps), q_start, lens)
    kw = dict(block_table=c.table, num_pool_blocks=c.pages)
    torch.cuda.synchronize()
    for _ in range(5):
        for p, ws, out, st in calls:
            with torch.cuda.stream(st):
                msa.msa_window_attn_q8(p, 900, 5, q, *args[0], *args[1:], out, ws, **kw)
    for p, ws, out, st in calls:
        msa.msa_workspace_status(ws, st)
        alone = torch.empty_like(out)
        msa.msa_window_attn_q8(p, 900, 5, q, *args[0], *args[1:], alone, ws, **kw)
        msa.msa_workspace_status(ws)
        assert torch.equal(out, alone)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kernels", ["streaming", "tensorcore"])
def test_pools_past_32_bits_of_offset(msa, kernels, q8):
    # the same few pages at the front of a small pool and at the end of one of
    # 4.6 GB: the same outputs, and the same bytes from the writer and the copy
    G, D, nb, T = 8, 128, 6, 33
    lens = [700, 333]
    c, q, q_start = make(lens, T, 16, G, D, seed=51, nb=nb)
    kv = list((*c.codes, *c.exps) if q8 else bf16_cache(c))
    page = kv[0][0].numel() * kv[0].element_size()
    pages = (4600 << 20) // page
    shift = pages - c.pages
    assert shift * page > 1 << 32
    big = []
    for x in kv:
        y = torch.empty((pages, *x.shape[1:]), dtype=x.dtype, device="cuda")
        y[shift:] = x
        big.append(y)
    p = msa.params(2, T, 16, G, D, 32, nb, kernels=kernels)
    ws = msa.window_workspace(p)
    fn = msa.msa_window_attn_q8 if q8 else msa.msa_window_attn
    outs = []
    for pool, table, n in [(kv, c.table, c.pages), (big, c.table + shift, pages)]:
        out = torch.empty_like(q)
        fn(p, 500, 9, q, *pool, q_start, lens, out, ws, block_table=table, num_pool_blocks=n)
        msa.msa_workspace_status(ws)
        outs.append(out)
    assert torch.equal(*outs)
    pw = msa.pages_workspace(pages)
    lists = [torch.tensor(x, dtype=torch.int32, device="cuda")
             for x in ([shift, shift + 1], [shift + 3, 5])]
    want = [y[[shift, shift + 1]].clone() for y in big]
    msa.msa_pages_copy(msa.pools(big), pages, *lists, pw)
    msa.msa_workspace_status(pw)
    for y, w in zip(big, want):
        assert torch.equal(y[[shift + 3, 5]].view(torch.uint8), w.view(torch.uint8))
    if not q8:
        return
    # the sparse call and the writer on the same pools (copied pages put back)
    for x, y in zip(kv, big):
        y[shift:] = x
    sel = torch.full((2, T, G, 16), -1, dtype=torch.int32, device="cuda")
    sel[..., 0], sel[..., 1] = 0, 2
    w8 = msa.q8_workspace(p)
    new = [torch.randn(2, T, G, D, device="cuda").to(torch.bfloat16) for _ in range(2)]
    ki_new = torch.randn(2, T, 32, device="cuda").to(torch.bfloat16)
    outs, kis = [], []
    for pool, table, n in [(kv, c.table, c.pages), (big, c.table + shift, pages)]:
        kw = dict(block_table=table, num_pool_blocks=n)
        out = torch.empty_like(q)
        msa.msa_sparse_attn_q8(p, q, *pool, sel, q_start, lens, out, w8, **kw)
        msa.msa_workspace_status(w8)
        ki = torch.zeros(n, 128, 32, dtype=torch.bfloat16, device="cuda")
        msa.msa_cache_append_q8(p, *new, ki_new, q_start, *pool, ki, w8, **kw)
        msa.msa_workspace_status(w8)
        outs.append(out)
        kis.append(ki)
    assert torch.equal(*outs)
    assert torch.equal(kis[0], kis[1][shift:])
    for x, y in zip(kv, big):
        assert torch.equal(x, y[shift:])


@pytest.mark.parametrize("kernels", KERNELS)
@pytest.mark.parametrize("D", [64, 128])
def test_output_aligned_to_16_bytes_only(msa, kernels, D):
    lens, T = [700, 400], 130
    c, q, q_start = make(lens, T, 6, 2, D, seed=57)
    nb = c.table.shape[1]
    want = run(msa, c, True, q, q_start, lens, nb, 300, 4, kernels)
    p = msa.params(2, T, 6, 2, D, 32, nb, kernels=kernels)
    ws = msa.window_workspace(p)
    raw = torch.full((q.numel() + 24,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = raw[8:8 + q.numel()].view(q.shape)
    assert out.data_ptr() % 32 == 16
    msa.msa_window_attn_q8(p, 300, 4, q, *c.codes, *c.exps, q_start, lens, out, ws,
                           block_table=c.table, num_pool_blocks=c.pages)
    msa.msa_workspace_status(ws)
    assert torch.equal(out, want)
    assert (raw[:8] == 7).all() and (raw[8 + q.numel():] == 7).all()
