"""Projections with adapters over a prompt's rows: a slot spans many blocks of 256 rows, its last one in part."""
import pytest
import torch

from tests.test_lora_gpu import Case, shape_of
from tests.test_lora_rings_gpu import compare

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("side", ["in", "out"])
@pytest.mark.parametrize("B,T,rank,ids", [(1, 8192, 16, [1]), (1, 2049, 128, [2]), (2, 4103, 64, [0, -1]),
                                          (3, 1000, 24, [-1, 2, 2]), (5, 513, 8, [0, 1, 0, 5, 2]), (1, 257, 72, [0])])
def test_many_rows_a_slot(side, B, T, rank, ids):
    c = Case(shape_of(n_slots=B, n_tokens=T), side, 3, rank, ids, seed=T + rank)
    c.ids = c.ids.clamp(max=2)
    y = c.run().clone()
    compare(c, y)
    assert torch.equal(c.run(), y)
