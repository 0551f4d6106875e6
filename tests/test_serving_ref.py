"""The plain implementations that the serving operators are tested against,
checked on the CPU: e4m3 rounding against torch's conversion, the 8-bit
writer's invariants, and that a planted mistake in a mask leaves the bound."""
import numpy as np
import pytest
import torch

from tests import serving_ref as sr


def test_e4m3_codes_match_torch():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(20000) * 10.0 ** rng.integers(-4, 3, 20000),
                        np.arange(0, 449, 0.5), 2.0 ** np.arange(-14.0, 9.0)])
    x = np.clip(np.concatenate([x, -x]), -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(sr.round_e4m3(x), want)
    back = sr.decode_e4m3(np.arange(256, dtype=np.uint8))
    ref = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(back, ref, equal_nan=True)


def test_append_in_pieces_keeps_every_value_within_a_step():
    # row by row, growing values: each kept value is within half a step of the
    # last scale plus what its earlier roundings cost
    rng = np.random.default_rng(1)
    new = rng.standard_normal((130, 2, 4)) * np.linspace(0.1, 50, 130)[:, None, None]
    new = torch.from_numpy(new).to(torch.bfloat16).double().numpy()
    codes, exps = np.zeros((2, 128, 2, 4), np.uint8), np.full((2, 2), 55, np.int8)
    for t in range(130):
        sr.append(codes, exps, new[t:t + 1], [1, 0], t)
    got = sr.decode_e4m3(codes) * np.exp2(exps.astype(float))[:, None, :, None]
    got = np.concatenate([got[1], got[0][:2]])
    step = np.concatenate([np.repeat(exps[1:2], 128, 0), np.repeat(exps[0:1], 2, 0)])
    tol = np.abs(new) * 2.0 ** -4 + 2.0 ** -9 * np.exp2(step.astype(float))[..., None]
    assert (np.abs(got - new) <= tol).all()


@pytest.mark.parametrize("window,sinks", [(5, 0), (5, 2), (200, 3)])
def test_bound_rejects_a_window_off_by_one(window, sinks):
    g = torch.Generator().manual_seed(3)
    q = torch.randn(1, 40, 2, 64, generator=g, dtype=torch.float64)
    k = [torch.randn(40, 1, 64, generator=g, dtype=torch.float64)]
    v = [torch.randn(40, 1, 64, generator=g, dtype=torch.float64)]
    want, bound = sr.attend_call(q, k, v, [0], sr.window_seen(40, window, sinks, "cpu"), 0.125,
                                 sr.U_BF16)
    sr.check(want.to(torch.bfloat16), want, bound)
    if window < 40:
        off, _ = sr.attend_call(q, k, v, [0], sr.window_seen(40, window + 1, sinks, "cpu"), 0.125,
                                sr.U_BF16)
        with pytest.raises(AssertionError):
            sr.check(off, want, bound)


def test_unseen_rows_never_matter():
    g = torch.Generator().manual_seed(4)
    q = torch.randn(1, 3, 1, 64, generator=g, dtype=torch.float64)
    k = torch.randn(200, 1, 64, generator=g, dtype=torch.float64)
    v = torch.randn(200, 1, 64, generator=g, dtype=torch.float64)
    seen = sr.window_seen(200, 10, 1, "cpu")
    want, _ = sr.attend_call(q, [k], [v], [100], seen, 1.0, sr.U_BF16)
    k2, v2 = k.clone(), v.clone()
    k2[1:91], v2[103:] = torch.nan, torch.inf
    got, _ = sr.attend_call(q, [k2], [v2], [100], seen, 1.0, sr.U_BF16)
    assert torch.equal(got, want)
