"""gdn_attend at the limits of its arguments: the widest windows, scales of nothing and next to nothing."""
import pytest
import torch

from tests.attn_ref import Case
from tests.test_attend_gpu import Run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 100, 2 ** 30, 2 ** 30 + 1])
@pytest.mark.parametrize("n_sink", [0, 3])
@pytest.mark.parametrize("sizes", [dict(T=1, H=8, Hk=2, D=128, page=16, past=[10, 0, 127, 500]),
                                   dict(T=20, H=8, Hk=2, D=64, page=16, past=[10, 0, 300]),
                                   dict(T=16, H=4, Hk=1, D=256, page=16, past=[10, 0, 300], tree=True)])
def test_windows_wider_than_any_cache(sizes, n_sink, window, dtype):
    r = Run(Case(dtype=dtype, window=window, n_sink=n_sink, **sizes))
    r.call()
    r.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -112, -(2.0 ** -114), 2.0 ** -140])
@pytest.mark.parametrize("rows", [1, 12])
def test_large_scores_under_a_small_scale(rows, scale, dtype):
    """Queries and keys of 2^53: scores of some 2^109, which a scale brings to some 10, to 1 or to nothing (2^-140 is below
    the smallest normal number)."""
    r = Run(Case(dtype=dtype, T=rows, H=8, Hk=2, D=64, page=16, past=[300, 5], scale=scale))
    big = 2.0 ** 53
    r.q, r.ks = r.q * big, [k * big for k in r.ks]
    r.gpu["q"], r.gpu["k"] = r.q.cuda(), r.gpu["k"] * big
    r.call()
    r.check()
