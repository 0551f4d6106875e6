"""The dense backward pass reads its preparation (statistics, units, counters) only behind
the wait for it: dQ's CTAs are in the launch of the KV-outer ones, which waits in its
beginning, and not in a launch of their own that the KV-outer one lets in."""
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


class Call:
    def __init__(self, msa, B, T, H, G, D, starts, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        mb = (max(starts) + T + 127) // 128
        bf = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)   # noqa: E731
        self.starts, self.lens = starts, [s + T for s in starts]
        self.q, self.dout = bf(B, T, H, D), bf(B, T, H, D)
        self.k, self.v = bf(B, mb, 128, G, D), bf(B, mb, 128, G, D)
        self.p = msa.params(B, T, H, G, D, 64, mb)
        self.out, self.lse = R.attn_forward(self.q, self.k, self.v, starts, self.p.scale)
        self.grads = [torch.empty_like(x) for x in (self.q, self.k, self.v)]

    def run(self, msa, ws):
        for x in self.grads:
            x.fill_(NAN)
        msa.msa_dense_attn_bwd(self.p, self.q, self.k, self.v, self.out, self.lse, self.dout,
                               self.starts, self.lens, *self.grads, ws)

    def check(self):
        want, bound = R.attn_backward(self.q, self.k, self.v, self.out, self.dout, self.starts,
                                      self.lens, self.p.scale)
        for i, what in enumerate(("dq", "dk", "dv")):
            got = self.grads[i]
            if i:
                own = torch.arange(got.shape[1] * 128, device="cuda") < torch.tensor(
                    self.lens, device="cuda")[:, None]
                got, w, e = (x.flatten(1, 2)[own] for x in (got, want[i], bound[i]))
                R.check(got, w, e, what)
            else:
                R.check(got, want[i], bound[i], what)


@pytest.mark.parametrize("kw,launches", [
    # statistics, units, the products; the sums of dQ's splits; of blocks in several pieces
    (dict(B=1, T=77, H=4, G=1, D=64, starts=[200]), 3),
    (dict(B=1, T=77, H=4, G=1, D=64, starts=[0]), 4),       # and the first positions' statistics
    (dict(B=1, T=100, H=4, G=1, D=128, starts=[2000]), 4),
    (dict(B=1, T=1200, H=16, G=1, D=128, starts=[500]), 5)])
def test_one_launch_for_the_products(msa, kw, launches):
    c = Call(msa, seed=1, **kw)
    ws = msa.dense_bwd_workspace(c.p)
    n = msa.msa_kernel_launch_count()
    c.run(msa, ws)
    assert msa.msa_kernel_launch_count() - n == launches
    msa.msa_workspace_status(ws)
    c.check()


def test_calls_in_turn_on_one_workspace(msa):
    """Long and short calls behind one another without a wait between them: none reads what
    the one before left in the workspace."""
    calls = [Call(msa, 1, 900, 16, 2, 128, [300], 1), Call(msa, 1, 77, 4, 1, 64, [0], 2),
             Call(msa, 2, 130, 8, 8, 128, [1, 700], 3), Call(msa, 1, 1500, 12, 4, 64, [0], 4)]
    ws = torch.empty(max(msa.msa_dense_bwd_workspace_bytes(c.p) for c in calls), dtype=torch.uint8,
                     device="cuda").fill_(0xFF)
    first = []
    for c in calls:
        c.run(msa, ws)
        msa.msa_workspace_status(ws)
        c.check()
        first.append([x.clone() for x in c.grads])
    for order in ([0, 1, 2, 3], [3, 1, 0, 2], [1, 2, 1, 0], [2, 3, 1, 1]):
        for _ in range(5):
            for i in order:
                calls[i].run(msa, ws)
        msa.msa_workspace_status(ws)
        for c, want in zip(calls, first):
            assert all(torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))
                       for a, b in zip(c.grads, want))
