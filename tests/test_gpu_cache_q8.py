"""The 8-bit cache: msa_cache_append_q8 bit for bit against the plain writer,
and the attention that reads it (msa_sparse_attn_q8, msa_forward_q8) against
64-bit attention of the same codes, within the bounds of serving_ref."""
import numpy as np
import pytest
import torch

from tests import serving_ref as sr

pytestmark = pytest.mark.gpu

KERNELS = ["streaming", "tensorcore", "auto"]


@pytest.fixture(scope="module")
def msa():
    assert torch.cuda.is_available()
    import block_sparse_attention_04_gb300 as m
    m.load()
    return m


def randq(*shape, seed=77):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)


# ------------------------------------------------------------------ writer --
def run_append(msa, calls, B, G, D, Di, nb, paged, seed, start_exp=None):
    """calls: list of (q_start, new K, new V as float [B][T][G][D]).  Every
    call is made on the device and by the plain writer; caches compared whole."""
    rng = np.random.default_rng(seed)
    npool = B * nb + (5 if paged else 0)
    perm = rng.permutation(npool) if paged else np.arange(npool)
    table = perm[:B * nb].reshape(B, nb).astype(np.int32)
    kc = rng.integers(0, 256, (2, npool, 128, G, D), dtype=np.uint8)      # anything in unused rows
    ex = rng.integers(-128, 128, (2, npool, G)).astype(np.int8)
    if start_exp is not None:
        ex[:] = start_exp
    ki = rng.integers(0, 1 << 16, (npool, 128, Di)).astype(np.uint16)
    dk, dv = (torch.from_numpy(kc[i].copy()).cuda() for i in (0, 1))
    de = [torch.from_numpy(ex[i].copy()).cuda() for i in (0, 1)]
    dki = torch.from_numpy(ki.view(np.int16).copy()).cuda()
    dtab = torch.from_numpy(table).cuda()
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    for q_start, kn, vn in calls:
        T = kn.shape[1]
        new = [bf16(x) for x in (kn, vn)]
        kin = rng.integers(0, 1 << 16, (B, T, Di)).astype(np.uint16)
        p = msa.params(B, T, G, G, D, Di, nb)
        msa.msa_cache_append_q8(p, new[0].cuda(), new[1].cuda(),
                                torch.from_numpy(kin.view(np.int16)).cuda(), q_start, dk, dv, de[0],
                                de[1], dki, ws, block_table=dtab if paged else None,
                                num_pool_blocks=npool if paged else 0)
        msa.msa_workspace_status(ws)
        for b in range(B):
            for i in (0, 1):
                sr.append(kc[i], ex[i], new[i][b].double().numpy(), table[b], q_start[b])
            for j in range(T):
                t = q_start[b] + j
                ki[table[b, t // 128], t % 128] = kin[b, j]
    for got, want in ((dk, kc[0]), (dv, kc[1])):
        got = got.cpu().numpy()
        nan = (got & 0x7F) == 0x7F          # a NaN code may carry either sign
        assert np.array_equal(nan, (want & 0x7F) == 0x7F)
        assert np.array_equal(got[~nan], want[~nan])
    assert np.array_equal(de[0].cpu().numpy(), ex[0])
    assert np.array_equal(de[1].cpu().numpy(), ex[1])
    assert np.array_equal(dki.cpu().numpy().view(np.uint16), ki)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("D,G,Di", [(128, 8, 64), (64, 1, 32), (64, 3, 64)])
def test_append_prefill_then_steps(msa, paged, D, G, Di):
    rng = np.random.default_rng(D + G)
    B = 3
    starts = [0, 100, 255]                     # a fresh block, inside one, its last row
    calls = [(starts, rng.standard_normal((B, 301, G, D)), rng.standard_normal((B, 301, G, D)) * 40)]
    pos = [s + 301 for s in starts]
    for step in range(3):                      # tokens that raise the exponent again and again
        f = 10.0 ** step
        calls.append((pos, rng.standard_normal((B, 1, G, D)) * f,
                      rng.standard_normal((B, 1, G, D)) / f))
        pos = [x + 1 for x in pos]
    run_append(msa, calls, B, G, D, Di, nb=6, paged=paged, seed=7, start_exp=-9)


def test_append_special_values(msa):
    G, D = 2, 64
    x = np.zeros((1, 12, G, D))
    x[0, 0, 0, :4] = [np.nan, np.inf, -np.inf, 3.0]
    x[0, 1, 1, 0] = 3.3e38                      # above 448 * 2^119: saturates
    x[0, 2, 0, 1] = 1e-40                       # subnormal in bf16
    x[0, 3, :, 5] = 448.0
    x[0, 4, 0, 6] = 450.0                       # one bf16 step above 448
    x[0, 5, 0, 7] = -1e-30
    zero = np.zeros((1, 5, G, D))
    tiny = np.full((1, 3, G, D), 1e-39)
    calls = [([0], x, zero.repeat(3, 1)[:, :12]), ([12], zero, zero + 2.0), ([17], tiny, tiny)]
    run_append(msa, calls, 1, G, D, 32, nb=2, paged=True, seed=8)
    # a block whose first values are all zero, then a large one
    run_append(msa, [([128], zero, tiny[:, :1].repeat(5, 1)), ([133], zero + 1e30, zero)], 1, G, D,
               32, nb=2, paged=False, seed=9)


def test_append_stored_exponents_at_their_ends(msa):
    rng = np.random.default_rng(11)
    x = rng.standard_normal((2, 2, 4, 128))
    for e in (-128, -126, 119, 127):            # before the call, block begun at row 1
        run_append(msa, [([1, 127], x, x * 1e3)], 2, 4, 128, 64, nb=2, paged=True, seed=12,
                   start_exp=e)


def test_append_long_chunk(msa):
    rng = np.random.default_rng(13)
    x = rng.standard_normal((1, 1500, 2, 128)) * np.exp2(rng.integers(-3, 4, (1, 1500, 1, 1)))
    run_append(msa, [([77], x, -x)], 1, 2, 128, 64, nb=13, paged=True, seed=14)


def test_append_writes_nothing_through_a_bad_table_entry(msa):
    B, G, D, nb = 2, 2, 64, 2
    for entry in (-1, 5, 1 << 30):
        table = torch.tensor([[0, entry], [2, 3]], dtype=torch.int32, device="cuda")
        kc = torch.full((5, 128, G, D), 9, dtype=torch.uint8, device="cuda")
        vc, ki = kc.clone(), torch.zeros(5, 128, 32, dtype=torch.bfloat16, device="cuda")
        ke = torch.zeros(5, G, dtype=torch.int8, device="cuda")
        ve = ke.clone()
        x = torch.ones(B, 1, G, D, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(256, dtype=torch.uint8, device="cuda")
        msa.msa_cache_append_q8(msa.params(B, 1, G, G, D, 32, nb), x, x,
                                torch.ones(B, 1, 32, dtype=torch.bfloat16, device="cuda"), [130, 6],
                                kc, vc, ke, ve, ki, ws, block_table=table, num_pool_blocks=5)
        with pytest.raises(msa.MsaError) as e:
            msa.msa_workspace_status(ws)
        assert e.value.status == -1
        changed = (kc != 9).flatten(2).any(-1).nonzero().tolist()
        assert changed == [[2, 6]]
        assert ki.abs().sum(-1).nonzero().tolist() == [[2, 6]]


# --------------------------------------------------------------- attention --
class Cache:
    """A paged 8-bit cache of B sequences.  Pages that no sequence uses and
    rows behind each context hold NaN codes."""

    def __init__(self, lens, G, D, nb, seed, exp_lo=-8, exp_hi=-3, rows=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        B = len(lens)
        self.pages = B * nb + 3
        self.table = torch.randperm(self.pages, generator=g, device="cuda")[:B * nb]
        self.table = self.table.reshape(B, nb).int()
        shape = (self.pages, 128, G, D)
        used = torch.zeros(self.pages, 128, dtype=torch.bool, device="cuda")
        for b, n in enumerate(lens):
            flat = torch.arange(nb * 128, device="cuda") < n
            used[self.table[b].long()] = flat.view(nb, 128)
        self.codes, self.exps = [], []
        for _ in range(2):
            x = torch.randn(shape, generator=g, device="cuda") * 60
            c = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            c[~used] = 0x7F
            self.codes.append(c)
            self.exps.append(torch.randint(exp_lo, exp_hi, (self.pages, G), generator=g,
                                           device="cuda", dtype=torch.int8))

    def values(self):
        r = []
        for c, e in zip(self.codes, self.exps):
            x = sr.dequant(c, e)
            r.append([sr.rows_of(x, self.table, b) for b in range(self.table.shape[0])])
        return r


def random_sel(B, T, G, q_start, seed, empty=()):
    rng = np.random.default_rng(seed)
    sel = np.full((B, T, G, 16), -1, np.int32)
    for b in range(B):
        for i in range(T):
            lb = (q_start[b] + i) // 128
            for g in range(G):
                if (b, i, g) in empty:
                    continue
                n = min(15, lb)
                ids = np.sort(np.append(rng.choice(lb, n, replace=False) if lb else [], lb))
                sel[b, i, g, :n + 1] = ids
    return torch.from_numpy(sel).cuda()


def run_sparse(msa, c, q, sel, q_start, lens, nb, Di, kernels="auto", scale=None, paged=True):
    B, T, H, D = q.shape
    G = c.codes[0].shape[2]
    p = msa.params(B, T, H, G, D, Di, nb, kernels=kernels, scale=scale)
    ws = msa.q8_workspace(p)
    ws.fill_(0xFF)                    # the library needs no cleared scratch
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    if paged:
        kv, kw = (*c.codes, *c.exps), dict(block_table=c.table, num_pool_blocks=c.pages)
    else:
        kv = [x[c.table.long().reshape(-1)].contiguous() for x in (*c.codes, *c.exps)]
        kw = {}
    msa.msa_sparse_attn_q8(p, q, *kv, sel, q_start, lens, out, ws, **kw)
    msa.msa_workspace_status(ws)
    return out


SPARSE = [
    # lens, T, H, G, D, Di
    ([1, 127, 128, 129, 2049, 5000], 1, 48, 8, 128, 64),
    ([9000], 1, 64, 4, 64, 32),
    ([700, 2600], 3, 16, 1, 128, 32),
    ([2500], 333, 12, 4, 128, 64),
    ([2433, 1130], 130, 10, 2, 64, 64),
    ([400], 400, 4, 4, 64, 32),
]


@pytest.mark.parametrize("kernels", KERNELS)
@pytest.mark.parametrize("lens,T,H,G,D,Di", SPARSE)
def test_sparse_q8(msa, kernels, lens, T, H, G, D, Di):
    B, nb = len(lens), max(-(-n // 128) for n in lens) + 1
    c = Cache(lens, G, D, nb, seed=B + T)
    g = torch.Generator(device="cuda").manual_seed(5)
    q = torch.randn(B, T, H, D, generator=g, device="cuda").to(torch.bfloat16)
    q_start = [n - T for n in lens]
    empty = {(0, 0, 0), (B - 1, T - 1, G - 1)} if T > 1 else set()
    sel = random_sel(B, T, G, q_start, 6, empty)
    out = run_sparse(msa, c, q, sel, q_start, lens, nb, Di, kernels)
    k, v = c.values()
    # weights round to bf16; the tensor-core kernels also keep one bf16 partial
    # per selected block: 2^-8 of A twice
    u = sr.U_BF16 if kernels == "streaming" else 2 * sr.U_BF16
    want, bound = sr.attend_call(q, k, v, q_start, sr.sel_seen(sel, nb * 128, "cuda"), D ** -0.5, u)
    sr.check(out, want, bound)
    for b, i, gg in empty:
        hpg = H // G
        assert (out[b, i, gg * hpg:(gg + 1) * hpg] == 0).all()


@pytest.mark.parametrize("kernels", KERNELS)
def test_sparse_q8_spread_exponents_and_negative_scale(msa, kernels):
    # blocks whose scales differ by up to 2^70: large weights on small values
    # and the other way round
    lens, T, H, G, D = [1900, 900], 2, 16, 2, 64
    c = Cache(lens, G, D, 15, seed=21, exp_lo=-60, exp_hi=-9)
    g = torch.Generator(device="cuda").manual_seed(20)
    c.exps[1] = torch.randint(-40, 30, c.exps[1].shape, generator=g, device="cuda", dtype=torch.int8)
    q = randq(2, T, H, D)
    q_start = [n - T for n in lens]
    sel = random_sel(2, T, G, q_start, 22)
    k, v = c.values()
    for scale in (3.0, -0.07):
        out = run_sparse(msa, c, q, sel, q_start, lens, 15, 32, kernels, scale=scale)
        want, bound = sr.attend_call(q, k, v, q_start, sr.sel_seen(sel, 15 * 128, "cuda"), scale,
                                     2 * sr.U_BF16)
        sr.check(out, want, bound)


@pytest.mark.parametrize("kernels", KERNELS)
@pytest.mark.parametrize("zero", ["first", "last", "most", "loud"])
def test_sparse_q8_blocks_of_zeros_keep_their_weight(msa, kernels, zero):
    # a block of zero values is stored with the smallest exponent; its weights
    # count in full beside blocks of ordinary (and of large) values.  "loud":
    # zeros under a large exponent (a block whose largest token was overwritten)
    lens, T, H, G, D = [1900, 700], 3, 12, 2, 128
    c = Cache(lens, G, D, 15, seed=27)
    page = c.table[0].long()
    pick = {"first": page[:1], "last": page[14:15], "most": page[1:14],
            "loud": page[4:6]}[zero]
    c.codes[1][pick] = c.codes[1][pick] & 0x7F
    c.codes[1][pick] = torch.where(c.codes[1][pick] == 0x7F, c.codes[1][pick], 0)
    c.exps[1][pick] = 40 if zero == "loud" else -126
    if zero != "loud":
        c.exps[1][page[3]] = 90
    q = randq(2, T, H, D)
    q_start = [n - T for n in lens]
    sel = random_sel(2, T, G, q_start, 28)
    k, v = c.values()
    for scale in (0.01, 0.5):
        out = run_sparse(msa, c, q, sel, q_start, lens, 15, 32, kernels, scale=scale)
        want, bound = sr.attend_call(q, k, v, q_start, sr.sel_seen(sel, 15 * 128, "cuda"), scale,
                                     2 * sr.U_BF16)
        sr.check(out, want, bound)


@pytest.mark.parametrize("e", [-128, -126, 119, 127])
def test_exponents_outside_the_range_read_as_its_ends(msa, e):
    lens, H, G, D = [300], 4, 2, 64
    c = Cache(lens, G, D, 3, seed=23)
    c.exps[0].fill_(-6)
    c.exps[1].fill_(e)
    c.codes[1] = torch.where(c.codes[1] == 0x7F, c.codes[1], c.codes[1] & 0x87)   # small values
    q = randq(1, 1, H, D)
    sel = random_sel(1, 1, G, [299], 24)
    out = run_sparse(msa, c, q, sel, [299], lens, 3, 32)
    c2 = Cache(lens, G, D, 3, seed=23)
    c2.codes, c2.exps = c.codes, [c.exps[0], c.exps[1].clamp(-126, 119)]
    out2 = run_sparse(msa, c2, q, sel, [299], lens, 3, 32)
    assert torch.equal(out, out2)
    k, v = c.values()
    want, bound = sr.attend_call(q, k, v, [299], sr.sel_seen(sel, 384, "cuda"), D ** -0.5, sr.U_BF16)
    # bf16 outputs keep 2^-134 at the small end
    sr.check(out, want, bound + 2.0 ** -133)


@pytest.mark.parametrize("kernels", KERNELS)
def test_sparse_q8_per_sequence_equals_paged(msa, kernels):
    lens, T, H, G, D = [1500, 1100], 5, 12, 4, 128
    c = Cache(lens, G, D, 12, seed=31)
    q = randq(2, T, H, D)
    q_start = [n - T for n in lens]
    sel = random_sel(2, T, G, q_start, 32)
    a = run_sparse(msa, c, q, sel, q_start, lens, 12, 64, kernels)
    b = run_sparse(msa, c, q, sel, q_start, lens, 12, 64, kernels, paged=False)
    assert torch.equal(a, b)


@pytest.mark.parametrize("kernels", KERNELS)
def test_forward_q8_selects_like_the_bf16_forward(msa, kernels):
    lens, T, H, G, D, Di, nb = [5000, 4300], 40, 48, 8, 128, 64, 41
    c = Cache(lens, G, D, nb, seed=41)
    g = torch.Generator(device="cuda").manual_seed(42)

    def grid(*shape):
        return torch.randint(-8, 9, shape, generator=g, device="cuda").to(torch.bfloat16) / 8
    q = torch.randn(2, T, H, D, generator=g, device="cuda").to(torch.bfloat16)
    qi, ki = grid(2, T, G, Di), grid(c.pages, 128, Di)
    q_start = [n - T for n in lens]
    p = msa.params(2, T, H, G, D, Di, nb, kernels=kernels)
    paged = dict(block_table=c.table, num_pool_blocks=c.pages)
    ws = msa.q8_workspace(p)
    sel = torch.empty(2, T, G, 16, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    msa.msa_forward_q8(p, qi, ki, q, *c.codes, *c.exps, q_start, lens, out, ws, sel_out=sel, **paged)
    msa.msa_workspace_status(ws)
    # the bf16 forward on the dequantised cache (exact in bf16; unused rows zero)
    kb = [torch.nan_to_num(sr.dequant(x, e)).to(torch.bfloat16) for x, e in zip(c.codes, c.exps)]
    ws2, sel2, out2 = msa.workspace(p), torch.empty_like(sel), torch.empty_like(out)
    msa.msa_forward_paged(p, c.table, c.pages, qi, ki, q, *kb, q_start, lens, out2, ws2,
                          sel_out=sel2)
    msa.msa_workspace_status(ws2)
    assert torch.equal(sel, sel2)
    k, v = c.values()
    want, bound = sr.attend_call(q, k, v, q_start, sr.sel_seen(sel, nb * 128, "cuda"), D ** -0.5,
                                 2 * sr.U_BF16)
    sr.check(out, want, bound)
    # without sel_out the selection lives in ws: same outputs
    out3 = torch.empty_like(out)
    msa.msa_forward_q8(p, qi, ki, q, *c.codes, *c.exps, q_start, lens, out3, ws, **paged)
    msa.msa_workspace_status(ws)
    assert torch.equal(out3, out)


@pytest.mark.parametrize("kernels", KERNELS)
def test_q8_bad_blocks_are_reported_and_skipped(msa, kernels):
    lens, T, H, G, D, nb = [900], 2, 4, 1, 64, 8
    c = Cache(lens, G, D, nb, seed=51)
    q = randq(1, T, H, D)
    q_start = [898]
    sel = random_sel(1, T, G, q_start, 52)
    good = sel.clone()
    sel[0, 0, 0, 2] = 8                      # beyond the local block
    good[0, 0, 0, 2] = -1
    p = msa.params(1, T, H, G, D, 32, nb, kernels=kernels)
    ws = msa.q8_workspace(p)
    out = torch.empty_like(q)
    paged = dict(block_table=c.table, num_pool_blocks=c.pages)

    def call(s, **kw):
        msa.msa_sparse_attn_q8(p, q, *c.codes, *c.exps, s, q_start, lens, out, ws, **{**paged, **kw})

    call(sel)
    with pytest.raises(msa.MsaError) as e:
        msa.msa_workspace_status(ws)
    assert e.value.status == -1
    bad = out.clone()
    call(good)
    msa.msa_workspace_status(ws)             # the next call starts from a clean status
    assert torch.equal(bad, out)
    table = c.table.clone()
    table[0, 3] = c.pages
    call(good, block_table=table)
    with pytest.raises(msa.MsaError) as e:
        msa.msa_workspace_status(ws)
    assert e.value.status == -1
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("kernels", KERNELS)
@pytest.mark.parametrize("T", [2, 200])
def test_a_block_listed_twice_counts_twice(msa, kernels, T):
    lens, H, G, D = [1500], 12, 4, 64
    nb = 13
    c = Cache(lens, G, D, nb, seed=61)
    q = randq(1, T, H, D)
    q_start = [1500 - T]
    rng = np.random.default_rng(62)
    sel = np.full((1, T, G, 16), -1, np.int32)
    for i in range(T):
        for g in range(G):
            lb = (q_start[0] + i) // 128
            ids = np.sort(np.append(rng.choice(lb, 6, replace=False), [lb]))
            sel[0, i, g, :9] = np.sort(np.append(ids, ids[[1, 3]]))
    sel = torch.from_numpy(sel).cuda()
    out = run_sparse(msa, c, q, sel, q_start, lens, nb, 32, kernels)
    k, v = c.values()
    # the reference holds every row twice; the second copy is visible where its
    # block is listed twice
    N = nb * 128
    block = torch.arange(N, device="cuda") // 128

    def seen(b, g, t):
        count = (sel[b, :, g, :, None] == torch.arange(nb, device="cuda")).sum(1)[:, block]
        causal = torch.arange(N, device="cuda") <= t[:, None]
        return torch.cat([(count > 0) & causal, (count > 1) & causal], 1)

    twice = [[torch.cat([x, x]) for x in y] for y in (k, v)]
    u = sr.U_BF16 if kernels == "streaming" else 2 * sr.U_BF16
    want, bound = sr.attend_call(q, *twice, q_start, seen, D ** -0.5, u)
    sr.check(out, want, bound)


def test_append_of_the_largest_batch(msa):
    # 256 sequences, one of them without room left behind it
    G, D, Di, nb = 2, 64, 32, 2
    c = Cache([0] * 256, G, D, nb, seed=63)
    g = torch.Generator(device="cuda").manual_seed(64)
    new = [torch.randn(256, 3, G, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    ki_new = torch.randn(256, 3, Di, generator=g, device="cuda").to(torch.bfloat16)
    ki = torch.zeros(c.pages, 128, Di, dtype=torch.bfloat16, device="cuda")
    q_start = [(i * 5) % 254 for i in range(255)] + [253]
    p = msa.params(256, 3, G, G, D, Di, nb)
    ws = msa.q8_workspace(p)
    msa.msa_cache_append_q8(p, *new, ki_new, q_start, *c.codes, *c.exps, ki, ws,
                            block_table=c.table, num_pool_blocks=c.pages)
    msa.msa_workspace_status(ws)
    for b, a in enumerate(q_start):
        for i in range(3):
            page, r = int(c.table[b, (a + i) // 128]), (a + i) % 128
            assert torch.equal(ki[page, r], ki_new[b, i])
            for x, codes, e in zip(new, c.codes, c.exps):
                got = sr.dequant(codes[page:page + 1], e[page:page + 1])[0, r]
                scale = torch.exp2(e[page].double())[:, None]
                bound = (x[b, i].double().abs() * 2.0 ** -4).maximum(scale * 2.0 ** -10)
                assert ((got.double() - x[b, i].double()).abs() <= bound).all()
