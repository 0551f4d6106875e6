"""The plain forms of the page workloads in perf/operators.py, on the CPU: their
results against a sequential host form, and no index assignment that names one
place twice with different values (its outcome would depend on the order of the
writes, which is undefined on a GPU)."""
import importlib.util
import os
import random

import numpy as np
import pytest
import torch
from torch.overrides import TorchFunctionMode

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf",
                    "operators.py")


@pytest.fixture()
def ops():
    spec = importlib.util.spec_from_file_location("workloads", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.DEV = "cpu"
    return m


class OneWriter(TorchFunctionMode):
    """Every x[index] = values writes each place of x once, or the same value."""

    def __torch_function__(self, func, types, args=(), kwargs=None):
        if func is torch.Tensor.__setitem__:
            x, index, value = args
            place = torch.arange(x.numel()).view(x.shape)[index].reshape(-1)
            v = torch.as_tensor(value, dtype=x.dtype).expand_as(x[index]).reshape(-1)
            order = place.argsort(stable=True)
            same = place[order][1:] == place[order][:-1]
            assert not (same & (v[order][1:] != v[order][:-1])).any(), "a place written twice"
        return func(*args, **(kwargs or {}))


def small(ops, op, seed):
    """A drawn case of the operator, in few and small pages."""
    rng = random.Random(seed)
    while True:
        c = ops.draw(rng)
        if c["op"] == op and c["pages"] < 400:
            return {**c, "H": 2, "G": 1, "D": 64, "Di": 32}


def host(s):
    return {k: (s[k].view(torch.int16) if s[k].dtype == torch.bfloat16 else s[k]).numpy().copy()
            for k in ("k", "v", "ki", "ke", "ve", "table", "refs") if s[k] is not None}


def same(got, want):
    for k, w in want.items():
        g = got[k]
        g = g.view({1: torch.uint8, 2: torch.int16}[g.element_size()]) if g.is_floating_point() else g
        assert np.array_equal(g.numpy(), w), k


@pytest.mark.parametrize("seed", range(6))
def test_compact(ops, seed):
    s = ops.prepare(small(ops, "compact", seed), seed)
    w = host(s)
    pages = len(w["refs"])
    live = int((w["refs"] > 0).sum())
    free = iter([i for i in range(live) if w["refs"][i] == 0])
    for i in range(live, pages):
        if w["refs"][i] > 0:
            h = next(free)
            for k in ("k", "v", "ki", "ke", "ve"):
                if k in w:
                    w[k][h] = w[k][i]
            w["table"][w["table"] == i] = h
            w["refs"][h], w["refs"][i] = w["refs"][i], 0
    with OneWriter():
        got = ops.run(s)
    same(got, w)
    assert got["live"].item() == live


@pytest.mark.parametrize("seed", range(6))
def test_fork(ops, seed):
    s = ops.prepare(small(ops, "fork", seed), seed)
    w = host(s)
    for a, b, n in zip(s["src"], s["dst"], s["lens"]):
        w["table"][b] = -1
        w["table"][b, :n // 128] = w["table"][a, :n // 128]
        np.add.at(w["refs"], w["table"][b, :n // 128], 1)
    for a, b, n in zip(s["src"], s["dst"], s["lens"]):
        if n % 128:
            old, new = w["table"][a, n // 128], np.flatnonzero(w["refs"] == 0)[0]
            w["table"][b, n // 128], w["refs"][new] = new, 1
            for k in ("k", "v", "ki"):
                w[k][new, :n % 128] = w[k][old, :n % 128]
            for k in ("ke", "ve"):
                if k in w:
                    w[k][new] = w[k][old]
    with OneWriter():
        got = ops.run(s)
    same(got, w)
