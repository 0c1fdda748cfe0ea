"""gdn_attend replayed hundreds of times with nothing between the launches, the same bits each time: the warps of a CTA
meet in every order, so an access that no wait orders would show.  The kernels of few rows (four copies of them in bf16),
and those in fp32 at each size of a block."""
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


def replay(r):
    r.call()
    first = r.got().clone()
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        for _ in range(20):
            r.call(stream=stream)
    for _ in range(20):
        r.out.fill_(77)
        graph.replay()
        assert torch.equal(first, r.got())
    r.check()


FEW = {
    "one token": dict(T=1, H=8, Hk=2, D=128, page=16, past=[4000, 77, 0]),
    "one token, small heads": dict(T=1, H=16, Hk=2, D=64, page=32, past=[9000, 300]),
    "one token, large heads": dict(T=1, H=24, Hk=4, D=256, page=64, past=[5000, 0, 129]),
    "32 rows": dict(T=8, H=8, Hk=2, D=128, page=128, past=[8000]),
    "window, sinks": dict(T=2, H=10, Hk=2, D=64, page=16, past=[2000, 130, 3, 700], window=300, n_sink=4),
    "window, sinks, large heads": dict(T=3, H=8, Hk=2, D=256, page=32, past=[3000, 130], window=500, n_sink=9),
    "tree": dict(T=16, H=4, Hk=2, D=128, page=16, past=[700, 0, 127], tree=True),
    "tree, small heads": dict(T=32, H=2, Hk=2, D=64, page=8, past=[1000, 31], tree=True),
    "tree, large heads": dict(T=7, H=4, Hk=1, D=256, page=16, past=[1500, 3], tree=True),
}


@pytest.mark.parametrize("name", FEW)
def test_few_rows(name):
    replay(Run(Case(**FEW[name])))


MANY = {
    "window, sinks": dict(T=40, H=8, Hk=2, D=64, page=32, past=[2000, 130], window=300, n_sink=4),
    "tree": dict(T=64, H=16, Hk=4, D=128, page=16, past=[700, 0, 127], tree=True),
    "window over tree": dict(T=64, H=8, Hk=2, D=256, page=16, past=[900, 20], tree=True, window=40, n_sink=3),
}


@pytest.mark.parametrize("name", MANY)
def test_many_rows(name):
    replay(Run(Case(**MANY[name])))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows", [8, 16, 32, 64])
def test_f32(rows, d):
    """Each size of a block: a ring of 2 to 6 buffers, filled again beside the softmax."""
    replay(Run(Case(dtype="f32", T=rows // 4, H=8, Hk=2, D=d, page=16, past=[3000, 5, 61])))


@pytest.mark.parametrize("sizes", [dict(T=2, H=8, Hk=2, D=128, page=16, past=[2000, 30], window=300, n_sink=4),
                                   dict(T=16, H=4, Hk=2, D=64, page=8, past=[1500, 30], tree=True),
                                   dict(T=100, H=4, Hk=2, D=128, page=32, past=[500, 30])])
def test_f32_forms(sizes):
    replay(Run(Case(dtype="f32", **sizes)))
