"""Projections with adapters over every ring of stages the GEMM forms (by its activation rows), every width of an
adapter's unit and both of its boxes of rank columns, against the 64-bit form."""
import pytest
import torch

from tests.test_lora_gpu import Case, shape_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def compare(c, y):
    """y against the 64-bit form: a sum of n fp32 products is off by at most n 2^-24 of the sum of their magnitudes
    (taken twice); h = scale A x enters B h with that error and its own rounding, at most 2^-16 of it; the output is
    rounded to bf16 once."""
    x, w, a, b = c.x.double(), c.w.double(), c.a.double(), c.b.double()
    K, T = x.shape[1], c.shape.n_tokens
    ref, err = x @ w.T, K * 2.0 ** -23 * (x.abs() @ w.abs().T)
    for s, i in enumerate(c.ids.tolist()):
        if i >= 0:
            rows = slice(s * T, (s + 1) * T)
            scale = float(c.scale[i])
            h, hm = scale * (x[rows] @ a[i].T), scale * (x[rows].abs() @ a[i].abs().T)
            ref[rows] += h @ b[i].T
            err[rows] += ((K + 2 * c.rank + 8) * 2.0 ** -23 * hm + 2.0 ** -16 * h.abs()) @ b[i].abs().T
    bad = ~((y.double() - ref).abs() <= 2.0 ** -8 * (ref.abs() + err) + err)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())


# rows 32 | 48, 60 | 96, 144 | 176 .. 300: a ring of 5 | 4 | 3 | 2 stages, the last by halves.  The input projection has a
# tile for most SMs and its K blocks go round the ring; the output projection splits K over a cluster.
@pytest.mark.parametrize("rank", [8, 32, 64, 72, 128])
@pytest.mark.parametrize("B,T", [(2, 16), (48, 1), (4, 15), (8, 12), (9, 16), (11, 16), (256, 1), (20, 15), (3, 100)])
@pytest.mark.parametrize("side", ["in", "out"])
def test_rings_and_units(side, B, T, rank):
    s = shape_of(n_slots=B, n_tokens=T, n_qk_heads=16, n_v_heads=48, d_k=128, d_v=128, n_embd=1544)
    c = Case(s, side, 5, rank, [(3 * i) % 6 - 1 if B > 3 else 4 - i for i in range(B)], seed=1000 * rank + B * T)
    y = c.run().clone()
    compare(c, y)
    for _ in range(8):
        assert torch.equal(c.run(), y)


@pytest.mark.parametrize("B,T,rank,embd", [(9, 16, 32, 264), (32, 16, 16, 2048)])
def test_the_results_that_repeated_launches_are_compared_with(B, T, rank, embd):
    kw = dict(n_qk_heads=16, n_v_heads=48, d_k=128, d_v=128) if embd > 264 else {}
    c = Case(shape_of(n_slots=B, n_tokens=T, n_embd=embd, **kw), "in", 4, rank, [i % 5 - 1 for i in range(B)])
    compare(c, c.run())
