"""The projection GEMM in the rings of stages that tests/test_proj_stages_gpu.py does not form: four stages (33 to 80
activation rows) and two that move by halves (more than 160), gone round many times with cold weights, against the
64-bit product; and a block of 256 rows with a part of another."""
import pytest
import torch

import gated_deltanet_verify_gb300 as gdn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def bound(x, w):
    """The 64-bit product, and how far fp32 sums of K products (K 2^-24 of their magnitudes, taken twice) and one bf16
    rounding may be off it."""
    ref = x.double() @ w.double().T
    err = x.shape[1] * 2.0 ** -23 * (x.double().abs() @ w.double().abs().T)
    return ref, 2.0 ** -8 * (ref.abs() + err) + err


@pytest.mark.parametrize("side", ["in", "out"])
@pytest.mark.parametrize("M", [48, 64, 80, 176, 240, 256, 272, 512])
def test_four_stages_and_two_by_halves(M, side):
    g = torch.Generator(device="cuda").manual_seed(M)
    heads, d, E = 48, 128, 2560
    dims = gdn.make_dims(M // 16, 16, heads, d, d, 16)
    n_in = 2 * 16 * d + 2 * heads * d + 2 * heads
    N, K = (n_in, E) if side == "in" else (E, heads * d)
    dummy = torch.zeros(8, dtype=torch.bfloat16, device="cuda")         # the other projection's weights: not read
    sets = []
    for _ in range(5):                                                  # more than 150 MB of weights: never all in L2
        w = (torch.randn((N, K), generator=g, device="cuda") * K ** -0.5).to(torch.bfloat16)
        x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
        sets.append((gdn.proj_weights(E, w, dummy) if side == "in" else gdn.proj_weights(E, dummy, w), x, w))
    call = gdn.gdn_project_in if side == "in" else gdn.gdn_project_out
    ld = gdn.gdn_proj_in_ld(dims) if side == "in" else E
    y, before = (torch.full((len(sets), M, ld), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for _ in range(60):
        for i, (weights, x, _) in enumerate(sets):
            call(dims, weights, x, before[i], None, 0)
    for i, (weights, x, _) in enumerate(sets):
        call(dims, weights, x, y[i], None, 0)
    torch.cuda.synchronize()
    for i, (_, x, w) in enumerate(sets):
        assert torch.equal(before[i, :, :N], y[i, :, :N])               # every launch gives the same bits
        ref, tol = bound(x, w)
        assert ((y[i, :, :N].double() - ref).abs() <= tol).all()
