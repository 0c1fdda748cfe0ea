"""Projections with low-rank adapters per slot against the plain 64-bit form, and the layer step that calls them."""
import numpy as np
import pytest
import torch

import gated_deltanet_verify_gb300 as gdn
from tests.gpu_util import dims_of, params_of, upload
from tests.step_ref import lora as lora_ref
from workloads.device import empty_outputs
from workloads.synth import Shape, make_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def shape_of(**kw):
    base = dict(name="lora", n_slots=3, n_qk_heads=2, n_v_heads=8, d_k=64, d_v=64, n_tokens=5, act="bf16", seed=91,
                n_embd=264)
    base.update(kw)
    return Shape(**base)


def columns(s):
    return s.conv_channels + s.value_dim + 2 * s.n_v_heads


class Case:
    """One projection's tensors; side "in" or "out"."""

    def __init__(self, shape, side, n, rank, ids, seed=0, scale=True):
        g = torch.Generator(device="cuda").manual_seed(seed)
        K, N = (shape.n_embd, columns(shape)) if side == "in" else (shape.value_dim, shape.n_embd)
        rand = lambda std, *sh: (torch.randn(sh, generator=g, device="cuda") * std).to(torch.bfloat16)  # noqa: E731
        self.shape, self.side, self.M, self.N, self.n, self.rank = shape, side, shape.n_slots * shape.n_tokens, N, n, rank
        self.x, self.w = rand(1.0, self.M, K), rand(K ** -0.5, N, K)
        self.a, self.b = rand(K ** -0.5, n, rank, K), rand(rank ** -0.5, n, N, rank)
        self.scale = (0.5 + torch.rand(n, generator=g, device="cuda")) if scale else None
        self.ids = torch.tensor(ids, dtype=torch.int32, device="cuda")
        other = torch.zeros((columns(shape) if side == "out" else shape.n_embd,
                             shape.n_embd if side == "out" else shape.value_dim), dtype=torch.bfloat16, device="cuda")
        self.weights = gdn.proj_weights(shape.n_embd, *((self.w, other) if side == "in" else (other, self.w)))
        self.keep = other
        self.lora = gdn.lora(n, rank, self.a, self.b, self.scale)
        self.dims = dims_of(shape)
        self.size = gdn.gdn_lora_workspace_bytes(self.dims, rank)
        self.space = torch.full((self.size,), 255, dtype=torch.uint8, device="cuda")      # NaN in every float
        self.y = torch.full((self.M * N + 64,), 9.0, dtype=torch.bfloat16, device="cuda")

    def run(self, status=None, **kw):
        f = gdn.gdn_project_in_lora if self.side == "in" else gdn.gdn_project_out_lora
        f(self.dims, self.weights, self.lora, self.ids, self.x, self.y, self.space, self.size, status, **kw)
        return self.y[:self.M * self.N].view(self.M, self.N)

    def plain(self):
        y = torch.empty((self.M, self.N), dtype=torch.bfloat16, device="cuda")
        f = gdn.gdn_project_in if self.side == "in" else gdn.gdn_project_out
        f(self.dims, self.weights, self.x, y, None, 0)
        return y

    def check(self):
        y = self.run()
        torch.cuda.synchronize()
        assert (self.y[self.M * self.N:] == 9.0).all()
        h = lambda t: t.double().cpu().numpy()  # noqa: E731
        scale = np.ones(self.n) if self.scale is None else h(self.scale)
        ref, bound = lora_ref(h(self.x), h(self.w), h(self.a), h(self.b), scale, self.ids.tolist(), self.shape.n_tokens)
        bad = np.abs(h(y) - ref) > bound
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist())


@pytest.mark.parametrize("side", ["in", "out"])
@pytest.mark.parametrize("rank", [8, 16, 24, 40, 64, 72, 128])
def test_ranks(side, rank):
    Case(shape_of(), side, 3, rank, [2, -1, 0], seed=rank).check()


@pytest.mark.parametrize("side", ["in", "out"])
@pytest.mark.parametrize("B,T,ids", [
    (1, 1, [0]), (1, 1, [-1]), (1, 16, [3]), (1, 17, [3]), (2, 16, [1, 1]), (4, 1, [3, 0, 0, 2]), (5, 3, [0, 1, 2, 3, -1]),
    (16, 1, list(range(4)) * 4), (33, 2, [i % 5 - 1 for i in range(33)]), (7, 40, [0, -1, 1, 1, 2, 3, 0]),
    (20, 15, [i % 4 for i in range(20)]), (3, 100, [2, 0, 1]), (300, 1, [i % 5 - 1 for i in range(300)]),
])
def test_batches(side, B, T, ids):
    Case(shape_of(n_slots=B, n_tokens=T), side, 4, 16, ids, seed=B * 100 + T).check()


@pytest.mark.parametrize("side", ["in", "out"])
@pytest.mark.parametrize("kw", [dict(n_embd=8), dict(n_embd=72), dict(n_embd=1024, n_qk_heads=16, n_v_heads=48, d_k=32, d_v=32),
                                dict(n_embd=136, d_k=32, d_v=32, n_v_heads=8), dict(n_embd=5120, n_tokens=16, n_slots=1)])
def test_layer_sizes(side, kw):
    s = shape_of(**kw)
    Case(s, side, 2, 16, [i % 2 for i in range(s.n_slots)], seed=s.n_embd, scale=False).check()


@pytest.mark.parametrize("side", ["in", "out"])
@pytest.mark.parametrize("kw", [{}, dict(n_embd=1024, n_qk_heads=16, n_v_heads=48, d_k=32, d_v=32, n_slots=9)])
def test_a_slot_without_an_adapter_is_the_shared_projection_bit_for_bit(side, kw):
    s = shape_of(**kw)
    c = Case(s, side, 2, 24, [-1 if i % 3 else 1 for i in range(s.n_slots)])
    got, base = c.run().clone(), c.plain()
    rows = torch.arange(c.M, device="cuda") // s.n_tokens % 3 != 0
    assert torch.equal(got[rows], base[rows])
    assert not torch.equal(got[~rows], base[~rows])
    c.b.zero_()
    assert torch.equal(c.run(), base)          # a term of zeros


def test_a_slot_does_not_see_its_neighbours():
    # slots that share groups of 16 rows: an infinite input, scale or A of one leaves the others' rows as they were
    s = shape_of(n_slots=6, n_tokens=5)
    c = Case(s, "in", 3, 16, [0, 1, 2, -1, 1, 0])
    want = c.run().clone()
    c.x[5:10] = float("inf")
    c.scale[2] = float("inf")
    c.a[2, 3] = float("nan")
    got = c.run()
    for slot in (0, 3, 4, 5):
        assert torch.equal(got[5 * slot:5 * slot + 5], want[5 * slot:5 * slot + 5]), slot
    assert not torch.isfinite(got[5:15].float()).any()


@pytest.mark.parametrize("bad", [-2, 3, 2 ** 31 - 1])
def test_an_unknown_adapter_is_reported_and_runs_without(bad):
    c = Case(shape_of(), "in", 3, 16, [0, bad, 2])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, base = c.run(status), c.plain()
    T = c.shape.n_tokens
    assert int(status) == gdn.GDN_ERR_ADAPTER
    assert torch.equal(got[T:2 * T], base[T:2 * T]) and not torch.equal(got[:T], base[:T])


def test_repeats_graphs_and_streams():
    c = Case(shape_of(n_slots=9, n_tokens=16), "in", 4, 32, [i % 5 - 1 for i in range(9)])
    want = c.run().clone()
    torch.cuda.synchronize()
    assert torch.equal(c.run(), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run()
    side.synchronize()
    assert torch.equal(c.y[:c.M * c.N].view(c.M, c.N), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
        c.run()                                # two in a row share the workspace in order
    c.y.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.y[:c.M * c.N].view(c.M, c.N), want)
    c.ids.copy_(torch.tensor([3] * 9, dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.y[:c.M * c.N].view(c.M, c.N), c.run())


def test_large_batches_back_to_back():
    # several launches at once in flight, each one's weights asked for while the one before ends
    c = Case(shape_of(n_slots=32, n_tokens=16, n_qk_heads=16, n_v_heads=48, d_k=128, d_v=128, n_embd=2048), "in", 4, 16,
             [i % 5 - 1 for i in range(32)])
    want, shared = c.run().clone(), c.plain()
    torch.cuda.synchronize()
    for _ in range(20):
        got = [c.plain(), c.plain()]
        c.run()
        c.run()
        got.append(c.plain())
    torch.cuda.synchronize()
    assert torch.equal(c.y[:c.M * c.N].view(c.M, c.N), want)
    assert all(torch.equal(y, shared) for y in got)


def _layer(shape, cases, which, x, status):
    """gdn_layer_verify_lora with adapters on the projections named in `which`; (y, act, out)."""
    dims = dims_of(shape)
    i, o = cases
    w = gdn.proj_weights(shape.n_embd, i.w, o.w)
    rank = max(c.rank for c, n in zip(cases, ("in", "out")) if n in which)
    size = gdn.gdn_layer_lora_workspace_bytes(dims, shape.n_embd, rank)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    y = torch.empty((i.M, shape.n_embd), dtype=torch.bfloat16, device="cuda")
    e = empty_outputs(shape, "cuda")
    gdn.gdn_layer_verify_lora(dims, params_of(x), w, i.lora if "in" in which else None, o.lora if "out" in which else None,
                              i.ids, i.x, x["state"], x["conv_state"], e["cap_state"], e["cap_conv"], y, ws, size, status)
    torch.cuda.synchronize()
    ld = gdn.gdn_proj_in_ld(dims)
    act = ws[:i.M * ld * 2].view(torch.bfloat16).view(i.M, ld)
    off = (i.M * ld * 2 + 255) // 256 * 256
    return y, act, ws[off:off + i.M * shape.value_dim * 2].view(torch.bfloat16).view(i.M, -1), e


@pytest.mark.parametrize("which", ["in", "out", "inout"])
def test_the_layer_is_its_three_steps_bit_for_bit(which):
    shape = shape_of()
    ids = [1, -1, 0]
    i, o = Case(shape, "in", 2, 16, ids, seed=1), Case(shape, "out", 2, 32, ids, seed=2)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    x, xs = upload(make_inputs(shape)), upload(make_inputs(shape))
    y, act, out, e = _layer(shape, (i, o), which, x, status)
    assert int(status) == 0
    want = (i.run() if "in" in which else i.plain()).clone()
    assert torch.equal(act[:, :i.N], want)
    C, V, H = shape.conv_channels, shape.value_dim, shape.n_v_heads
    a = want.view(shape.n_slots, shape.n_tokens, -1)
    part = [a[:, :, p:q].contiguous() for p, q in ((0, C), (C, C + V), (C + V, C + V + H), (C + V + H, C + V + 2 * H))]
    f = empty_outputs(shape, "cuda")
    gdn.gdn_verify_forward(dims_of(shape), params_of(xs), *part, xs["state"], xs["conv_state"], f["cap_state"],
                           f["cap_conv"], f["out"], None)
    assert torch.equal(f["out"].view(out.shape), out) and torch.equal(xs["state"], x["state"])
    assert torch.equal(e["cap_state"], f["cap_state"]) and torch.equal(e["cap_conv"], f["cap_conv"])
    o.x = out.contiguous()
    assert torch.equal(y, o.run() if "out" in which else o.plain())
