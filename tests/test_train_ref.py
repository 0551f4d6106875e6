"""The plain training pass of tests/train_ref.py against central differences and
against torch's own differentiation (no GPU)."""
import math

import pytest
import torch

from tests import train_ref as R


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_gradient(interleaved):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(2, 3, 2, 64, generator=g, dtype=torch.float64)
    w = torch.randn(64, generator=g, dtype=torch.float64)
    dy = torch.randn(x.shape, generator=g, dtype=torch.float64)
    t = torch.tensor([[5, 6, 7], [100000, 100001, 100002]])
    f = [10000.0 ** (-i / 16) for i in range(16)]

    def fn(x, w):
        return R.norm_rope(x, w, t, f, interleaved, 1.2, 1e-6)[0]

    dx, _, dw, _ = R.norm_rope_bwd(x, w, dy, t, f, interleaved, 1.2, 1e-6)
    for _ in range(4):
        at = torch.randn(x.shape, generator=g, dtype=torch.float64)
        want = R.finite_difference(lambda y: fn(y, w), x, dy, at)
        assert abs((dx * at).sum().item() - want) < 1e-5 * (1 + abs(want))
        aw = torch.randn(w.shape, generator=g, dtype=torch.float64)
        want = R.finite_difference(lambda y: fn(x, y), w, dy, aw)
        assert abs((dw * aw).sum().item() - want) < 1e-5 * (1 + abs(want))


def test_rotation_keeps_relative_positions():
    g = torch.Generator().manual_seed(2)
    a, b = (torch.randn(1, 1, 1, 64, generator=g, dtype=torch.float64) for _ in range(2))
    f = [10000.0 ** (-i / 32) for i in range(32)]
    dots = [(R.rotate(a, torch.tensor([[t + 7]]), f, False, 1.0) *
             R.rotate(b, torch.tensor([[t]]), f, False, 1.0)).sum() for t in (0, 1000, 123456)]
    assert max(dots) - min(dots) < 1e-9


@pytest.mark.parametrize("sparse", [False, True])
def test_attention_gradient(sparse):
    g = torch.Generator().manual_seed(3)
    T, H, G, D, q0 = 40, 4, 2, 64, 250
    N = q0 + T
    q = torch.randn(1, T, H, D, generator=g, dtype=torch.float64)
    k, v = (torch.randn(1, 3, 128, G, D, generator=g, dtype=torch.float64) for _ in range(2))
    dout = torch.randn(1, T, H, D, generator=g, dtype=torch.float64)
    sel = None
    if sparse:
        sel = R.random_sel(T, G, [q0], g, "cpu")
        sel[0, 3, 0] = torch.tensor([2, 2, 1] + [-1] * 13)      # an id twice
        sel[0, 4, 1] = -1                                        # none
        sel[0, 5, 1] = 0
        sel[0, 6, 0, 1] = 7                                      # past the local block
    out, _ = R.attn_forward(q, k, v, [q0], 0.3, sel)
    (dq, dk, dv), _ = R.attn_backward(q, k, v, out, dout, [q0], [N], 0.3, sel)
    x = [z.clone().requires_grad_() for z in (q, k, v)]
    total = 0
    for h in range(H):
        gi = h // (H // G)
        cnt = R.counts_dense(T, N, q0, "cpu") if sel is None else R.counts_sel(sel[0, :, gi], N, q0)
        some = cnt.sum(-1) > 0
        s = torch.where(cnt > 0, x[0][0, :, h] @ x[1][0].flatten(0, 1)[:N, gi].T * 0.3 +
                        torch.log(cnt.clamp(min=1)), -math.inf)[some]
        o = torch.softmax(s, -1) @ x[2][0].flatten(0, 1)[:N, gi]
        total = total + (o * dout[0, some, h]).sum()
    want = torch.autograd.grad(total, x)
    for a, b in zip((dq, dk, dv), want):
        assert (a - b).abs().max() < 1e-12
