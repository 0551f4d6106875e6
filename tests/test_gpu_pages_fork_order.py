"""The order of msa_pages_fork that msa.h states: all destination rows let go of
their pages before free pages are handed out, lowest first, in order of the pairs."""
import pytest
import torch

from tests.test_gpu_pages import contiguous_world

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def msa():
    assert torch.cuda.is_available()
    import block_sparse_attention_04_gb300 as m
    m.load()
    return m


def test_pages_of_later_destination_rows_are_free_for_the_first_pair(msa):
    # a full pool: the only free pages are those that the last destination row held
    w = contiguous_world(9, 5, 4, [300, 200, 0, 0, 500], seed=6)
    assert (w.refs == 1).all()
    w.device(msa)
    src, dst, lens = [0, 1, 1], [2, 3, 4], [300, 129, 200]
    msa.msa_pages_fork(w.set, 9, w.d_table, w.d_refs, src, dst, lens, w.ws)
    msa.msa_workspace_status(w.ws)
    let_go = sorted(w.table[4].tolist())
    w.fork(src, dst, lens)
    assert [w.table[2, 2], w.table[3, 1], w.table[4, 1]] == let_go[:3]
    w.same()
