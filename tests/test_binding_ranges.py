"""Host integers that do not fit 32 bits, which the C ABI cannot take: windows and
sink counts keep their meaning (a window of at least the context is dense), and
positions, lengths, rows and block ranges are refused.  No GPU: the calls go to a
recorder or are refused before the library."""
import numpy as np
import pytest
import torch

import block_sparse_attention_04_gb300 as msa

PTR = 0x10000


class Recorder:
    """Stands for the library: keeps the arguments of the last call."""

    def __getattr__(self, name):
        def call(*args):
            self.args = args
            return 0
        return call


@pytest.fixture()
def rec(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(msa, "load", lambda path=None: r)
    return r


class Ws:
    nbytes = 1 << 30


@pytest.mark.parametrize("given,passed", [
    (1, 1), ((1 << 31) - 1, (1 << 31) - 1), (1 << 31, (1 << 31) - 1), ((1 << 32) + 5, (1 << 31) - 1),
    (1 << 40, (1 << 31) - 1), (1 << 70, (1 << 31) - 1), (-3, -1), (-(1 << 32) + 5, -1)])
@pytest.mark.parametrize("q8", [False, True])
def test_windows_and_sinks(rec, monkeypatch, given, passed, q8):
    monkeypatch.setattr(msa, "_ptr", lambda t: None if isinstance(t, Ws) else t)
    p = msa.params(1, 1, 4, 2, 64, 32, 8)
    fn = msa.msa_window_attn_q8 if q8 else msa.msa_window_attn
    kv = [PTR] * (4 if q8 else 2)
    fn(p, given, 7, PTR, *kv, [0], [1], PTR, Ws(), stream=0)
    assert rec.args[3:5] == (passed, 7)
    fn(p, 9, given, PTR, *kv, [0], [1], PTR, Ws(), stream=0)
    assert rec.args[3:5] == (9, passed)


@pytest.mark.parametrize("make", [list, tuple, lambda x: np.array(x, dtype=np.int64),
                                  lambda x: [float(v) for v in x], torch.tensor])
@pytest.mark.parametrize("big", [1 << 31, -(1 << 31) - 1, 1 << 32, (1 << 40) + 3])
def test_positions_past_32_bits_are_refused(make, big):
    with pytest.raises(ValueError, match="32 bits"):
        msa.positions(make([5, big]))
    with pytest.raises(ValueError, match="32 bits"):
        msa._host_i32(make([big, 5]), 2)
    ends = [(1 << 31) - 1, -(1 << 31), 0]
    assert list(msa.positions(make(ends))) == ends


def test_block_ranges_past_32_bits_are_refused(rec):
    table, refs = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    ws = torch.zeros(4096, dtype=torch.uint8)
    for fn in (msa.msa_pages_free, msa.msa_pages_alloc):
        with pytest.raises(ValueError, match="32 bits"):
            fn(3, table, refs, [0], [0], [1 << 32], ws, stream=0)
    d = msa.pools([torch.zeros(3, 128, 2, dtype=torch.int16)])
    with pytest.raises(ValueError, match="32 bits"):
        msa.msa_pages_fork(d, 3, table, refs, [0], [1], [(1 << 32) + 130], ws, stream=0)
    assert "args" not in vars(rec)
    msa.msa_pages_free(3, table, refs, [], [], [], ws, stream=0)      # empty lists are fine
    assert rec.args[8] == 0


def test_a_scalar_stands_for_every_sequence():
    assert list(msa._host_i32(7, 3)) == [7, 7, 7]
    with pytest.raises(ValueError):
        msa._host_i32([1, 2], 3)
