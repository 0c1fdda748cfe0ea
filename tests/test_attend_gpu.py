"""gdn_attend against plain 64-bit sums: chains, trees, windows, chunks, pages in any order, NaN wherever nothing may look."""
import threading

import pytest
import torch

import gated_deltanet_verify_gb300 as gdn
from tests.attn_ref import NAN, Case, attend_bound, attend_ref, fill_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


class Run:
    """A case's buffers on the GPU."""

    def __init__(self, c):
        self.c = c
        c.pages()
        self.kp, self.vp, self.ks, self.vs = fill_cache(c)
        self.q = c.rand(c.B, c.T, c.H, c.D, std=1.5)
        self.parent = c.parents() if c.tree else None
        for s in range(c.B):
            self.q[s, c.n(s):] = NAN
        self.dims = c.dims()
        self.params = gdn.attn_params(c.scale, c.window, c.n_sink)
        self.gpu = {k: v.cuda() for k, v in dict(k=self.kp, v=self.vp, table=c.table, q=self.q,
                                                past=torch.tensor(c.past, dtype=torch.int32)).items()}
        self.length = torch.tensor(c.length, dtype=torch.int32).cuda() if c.length is not None else None
        self.d_parent = self.parent.cuda() if c.tree else None
        self.size = gdn.gdn_attend_workspace_bytes(self.dims)
        self.space = torch.full((self.size + 256,), 0xFF, dtype=torch.uint8, device="cuda")      # NaN as floats
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.out = torch.full((c.B * c.T * c.H * c.D + 64,), 77.0, dtype=c.dtype, device="cuda")

    def call(self, out=None, stream=None):
        g = self.gpu
        cache = gdn.kv_cache(g["k"], g["v"], g["table"], g["past"])
        gdn.gdn_attend(self.dims, cache, self.params, g["q"], self.out if out is None else out, self.space, self.size,
                       d_length=self.length, d_parent=self.d_parent, d_status=self.status, stream=stream)

    def got(self, out=None):
        torch.cuda.synchronize()
        c, o = self.c, (self.out if out is None else out).cpu()
        assert (o[c.B * c.T * c.H * c.D:] == 77).all()
        assert (self.space[self.size:] == 0xFF).all()
        return o[:c.B * c.T * c.H * c.D].view(c.B, c.T, c.H, c.D)

    def check(self, out=None, status=0):
        c, got = self.c, self.got(out).double()
        assert int(self.status.item()) == status
        for s, r in enumerate(attend_ref(c, self.q, self.ks, self.vs, self.parent)):
            n = c.n(s)
            assert (got[s, n:] == 77).all()
            if r is None:
                continue
            want, size, reach = r
            off = (got[s, :n] - want).abs() - attend_bound(c, s, want, size, reach)
            assert not got[s, :n].isnan().any() and float(off.max()) <= 0, (s, float(off.max()))


CASES = {
    "one token, empty cache": dict(T=1, H=4, Hk=4, D=64, page=8, past=[0]),
    "one token, one before": dict(T=1, H=6, Hk=1, D=256, page=16, past=[1]),
    "lengths about a tile": dict(T=1, H=8, Hk=2, D=128, page=16, past=[126, 127, 128, 129, 30, 31, 32, 33]),
    "lengths about a page": dict(T=3, H=8, Hk=2, D=128, page=8, past=[4, 5, 6, 7, 8, 9]),
    "verify": dict(T=16, H=24, Hk=4, D=256, page=64, past=[1000, 3, 517]),
    "verify, no past": dict(T=16, H=24, Hk=4, D=256, page=64, past=[0, 0]),
    "ragged": dict(T=7, H=12, Hk=4, D=128, page=32, past=[300, 0, 40, 999, 12, 0], length=[7, 1, 0, 3, 6, 0]),
    "all empty": dict(T=4, H=4, Hk=2, D=64, page=16, past=[5, 9], length=[0, 0]),
    "odd group": dict(T=5, H=35, Hk=5, D=64, page=16, past=[77, 200]),
    "group of 64": dict(T=3, H=64, Hk=1, D=128, page=128, past=[500, 20]),
    "group of 48": dict(T=6, H=48, Hk=1, D=64, page=256, past=[500, 20]),
    "no sharing": dict(T=9, H=5, Hk=5, D=128, page=256, past=[300, 2]),
    "page of 256": dict(T=2, H=8, Hk=2, D=256, page=256, past=[255, 256, 257, 700]),
    "page of 8, long": dict(T=4, H=8, Hk=2, D=256, page=8, past=[2049, 60]),
    "gap between pages": dict(T=4, H=8, Hk=2, D=128, page=16, past=[100, 3], gap=8 * 13),
    "chunk": dict(T=300, H=6, Hk=1, D=256, page=32, past=[0, 333]),
    "chunk, ragged": dict(T=150, H=8, Hk=2, D=128, page=64, past=[130, 5, 1000], length=[150, 1, 97]),
    "chunk, small heads": dict(T=257, H=3, Hk=3, D=64, page=16, past=[511]),
    "wide rows": dict(T=64, H=16, Hk=2, D=64, page=16, past=[700]),
    "tree": dict(T=16, H=24, Hk=4, D=256, page=16, past=[0, 127, 500], tree=True),
    "tree of 64": dict(T=64, H=8, Hk=2, D=128, page=32, past=[120, 0, 1000], tree=True, length=[64, 33, 2]),
    "tree of 64, wide": dict(T=64, H=40, Hk=5, D=64, page=8, past=[90], tree=True),
    "tree of one": dict(T=1, H=4, Hk=2, D=128, page=16, past=[9, 0], tree=True),
    "window": dict(T=1, H=8, Hk=2, D=128, page=16, past=[1000, 100, 99, 0], window=100),
    "window of one": dict(T=4, H=8, Hk=2, D=64, page=16, past=[300, 0], window=1),
    "window, sinks": dict(T=5, H=8, Hk=2, D=128, page=16, past=[2000, 130, 3, 700], window=64, n_sink=4),
    "window, many sinks": dict(T=2, H=8, Hk=2, D=256, page=32, past=[2000, 300, 40], window=33, n_sink=200),
    "window over chunk": dict(T=280, H=6, Hk=1, D=128, page=32, past=[100, 1500], window=50, n_sink=1),
    "window of one over chunk": dict(T=200, H=2, Hk=1, D=256, page=8, past=[10], window=1, n_sink=0),
    "window larger than all": dict(T=8, H=4, Hk=1, D=64, page=16, past=[50], window=2 ** 31 - 1, n_sink=2 ** 31 - 1),
    "window over tree": dict(T=40, H=6, Hk=2, D=128, page=16, past=[0, 200, 1000], window=7, n_sink=3, tree=True),
    "window over tree, no sinks": dict(T=64, H=6, Hk=2, D=64, page=16, past=[3, 130], window=2, tree=True),
    "many slots": dict(T=2, H=8, Hk=2, D=64, page=16, past=[(37 * i) % 400 for i in range(170)]),
    "more slots than a warp looks through": dict(T=1, H=4, Hk=2, D=128, page=8, past=[(91 * i) % 300 for i in range(300)]),
    "more blocks than a warp looks through": dict(T=1100, H=32, Hk=1, D=64, page=64, past=[40]),
    "one slot, long": dict(T=16, H=6, Hk=1, D=256, page=64, past=[13001]),
    "one slot, longer": dict(T=1, H=8, Hk=2, D=128, page=128, past=[26000]),
    "one slot, small heads, long": dict(T=2, H=8, Hk=4, D=64, page=16, past=[50011]),
    "three slots, one long": dict(T=4, H=8, Hk=4, D=128, page=32, past=[25000, 7, 300], length=[3, 4, 0]),
    "one long, many short": dict(T=1, H=8, Hk=2, D=128, page=64, past=[9000] + [i % 50 for i in range(40)]),
    "large scores": dict(T=3, H=4, Hk=2, D=64, page=16, past=[300], scale=6.0),
    "negative scale": dict(T=3, H=4, Hk=2, D=128, page=16, past=[300], scale=-0.2),
    "scale of zero": dict(T=3, H=4, Hk=2, D=128, page=16, past=[140], scale=0.0),
}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", CASES)
def test_cases(name, dtype):
    r = Run(Case(dtype=dtype, **CASES[name]))
    r.call()
    r.check()


# a slot's rows at and past each size of a block, its keys shared out among many CTAs and in one
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 7, 8, 9, 16, 17, 31, 32, 33, 64, 65])
def test_rows_of_a_block(rows, d, dtype):
    T, G = next((rows // g, g) for g in (5, 4, 3, 2, 1) if rows % g == 0)
    r = Run(Case(dtype=dtype, T=T, H=2 * G, Hk=2, D=d, page=16, past=[5000, 0, 61], length=[T, T, T - T // 2]))
    r.call()
    r.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_twice_the_same_bits(dtype):
    r = Run(Case(dtype=dtype, T=16, H=24, Hk=4, D=256, page=64, past=[3000, 3, 517]))
    r.call()
    first = r.got().clone()
    r.call()
    assert torch.equal(first, r.got())
    r.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_bad_lengths_skip_their_slots(dtype):
    c = Case(dtype=dtype, T=4, H=8, Hk=2, D=128, page=16, past=[200, 50, 20, 30])
    r = Run(c)
    room = c.max_pages * c.page
    want = r.out.clone()
    r.call(out=want)
    assert int(r.status.item()) == 0
    want = r.got(want)
    for past, length in ((-1, 4), (room - 3, 4), (2 ** 31 - 1, 4), (50, 5), (50, -1), (-2 ** 31, 4)):
        r.gpu["past"][1] = past
        r.length = torch.tensor([4, length, 4, 4], dtype=torch.int32, device="cuda")
        r.out.fill_(77)
        r.status.zero_()
        r.call()
        got = r.got()
        assert int(r.status.item()) == gdn.GDN_ERR_LENGTH, (past, length)
        assert (got[1] == 77).all()
        for s in (0, 2, 3):
            assert torch.allclose(got[s].float(), want[s].float(), rtol=2 ** -6, atol=2 ** -6)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("page", [8, 64, 256])
def test_bad_pages_read_as_zeros(dtype, page):
    c = Case(dtype=dtype, T=3, H=8, Hk=2, D=128, page=page, past=[600, 300])
    r = Run(c)
    for s, i, id in ((0, 1, -1), (1, 0, c.n_pages), (0, 0, 2 ** 31 - 1)):
        r.gpu["table"][s, i] = id
        for x in (r.ks, r.vs):
            x[s][i * page:(i + 1) * page] = 0
    r.call()
    r.check(status=gdn.GDN_ERR_PAGE)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_bad_parents_hang_from_the_past(dtype):
    c = Case(dtype=dtype, T=12, H=8, Hk=2, D=64, page=16, past=[40, 0], tree=True)
    r = Run(c)
    bad = r.parent.clone()
    for s, t, p in ((0, 3, 3), (0, 5, 100), (1, 2, -2), (1, 0, 0), (1, 7, -2 ** 31)):
        bad[s, t] = p
        r.parent[s, t] = -1
    r.d_parent = bad.cuda()
    r.call()
    r.check(status=gdn.GDN_ERR_TREE)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_what_no_token_sees_does_not_matter(dtype):
    """Below a window and behind the sinks: NaN in the pages' rows, junk ids for pages that hold nothing seen."""
    c = Case(dtype=dtype, T=3, H=8, Hk=2, D=128, page=16, past=[1000, 777], window=70, n_sink=5)
    r = Run(c)
    want = attend_ref(c, r.q, r.ks, r.vs)
    for s in range(c.B):
        low = c.past[s] - c.window + 1
        for p in range(c.n_sink, low):
            page, at = c.where(s, p)
            c.rows(r.kp)[page, :, at] = float("inf")
            c.rows(r.vp)[page, :, at] = NAN
        for i in range(1, low // c.page):
            r.gpu["table"][s, i] = (-5, c.n_pages + 9)[i % 2]
    r.gpu["k"], r.gpu["v"] = r.kp.cuda(), r.vp.cuda()
    r.call()
    r.check()
    assert len(want) == c.B


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_captured_with_changing_lengths(dtype):
    """One graph for every step: the lengths and pages are read on the device."""
    c = Case(dtype=dtype, T=4, H=8, Hk=2, D=128, page=16, past=[700, 20, 333])
    r = Run(c)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        r.call(stream=stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        r.call(stream=stream)
    for past in ([700, 20, 333], [10, 19, 0], [500, 3, 332]):
        c.past = past
        r.gpu["past"].copy_(torch.tensor(past, dtype=torch.int32))
        keep = r.ks, r.vs
        r.ks, r.vs = [k[:p + c.T] for k, p in zip(r.ks, past)], [v[:p + c.T] for v, p in zip(r.vs, past)]
        r.out.fill_(77)
        graph.replay()
        r.check()
        r.ks, r.vs = keep


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_two_streams_with_their_own_workspaces(dtype):
    runs = [Run(Case(dtype=dtype, T=5, H=24, Hk=4, D=128, page=32, past=[900 + 100 * i, 77], seed=i)) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(20):
        for r, s in zip(runs, streams):
            r.call(stream=s)
    for r in runs:
        r.check()


@pytest.mark.parametrize("sizes", [dict(T=16, H=32, Hk=8, D=128, page=128, past=[8000]),
                                   dict(T=16, H=24, Hk=4, D=256, page=64, past=[5000]),
                                   dict(T=40, H=8, Hk=4, D=64, page=64, past=[9000, 300])])
def test_launch_after_launch(sizes):
    """Hundreds of launches with nothing between them: the warps of a CTA meet in every order."""
    r = Run(Case(**sizes))
    r.call()
    first = r.got().clone()
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        for _ in range(20):
            r.call(stream=stream)
    for _ in range(20):
        graph.replay()
    assert torch.equal(first, r.got())
    r.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_host_threads(dtype):
    """Several host threads, each with its own stream, buffers and shape of kernel."""
    shapes = [dict(T=1, H=8, Hk=2, D=64, page=16, past=[900, 4]), dict(T=16, H=24, Hk=4, D=256, page=64, past=[1000]),
              dict(T=5, H=8, Hk=2, D=128, page=32, past=[700, 70]), dict(T=2, H=6, Hk=1, D=256, page=16, past=[300])]
    runs = [Run(Case(dtype=dtype, seed=i, **x)) for i, x in enumerate(shapes)]
    torch.cuda.synchronize()
    failed = []

    def work(r):
        try:
            torch.cuda.set_device(0)
            stream = torch.cuda.Stream()
            for _ in range(50):
                r.call(stream=stream)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(r,)) for r in runs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for r in runs:
        r.check()


def test_far_pages():
    """Pages whose offset in the pool passes 2^31 elements (and their bytes 2^32)."""
    c = Case(T=2, H=2, Hk=1, D=256, page=256, past=[300, 1000])
    r = Run(c)
    far = 2 ** 31 // (256 * 256) + 5
    pools = {}
    for name, flat in (("k", r.kp), ("v", r.vp)):
        big = torch.empty((far + c.n_pages, flat.shape[1]), dtype=c.dtype, device="cuda")
        big[far:] = flat.cuda()
        pools[name] = big
    r.gpu.update(pools)
    r.gpu["table"] = torch.where(c.table >= 0, c.table + far, -1).to(torch.int32).cuda()
    r.gpu["table"][c.table == 2 ** 31 - 1] = -1
    r.dims.n_pages = far + c.n_pages
    r.call()
    r.check()
