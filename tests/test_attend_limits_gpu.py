"""gdn_attend at the limits of its arguments: the widest windows."""
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
