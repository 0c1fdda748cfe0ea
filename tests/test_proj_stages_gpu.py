"""The projection GEMM where its ring of stages has an odd length and is gone round many times: repeated launches with
cold weights against the 64-bit product."""
import pytest
import torch

import gated_deltanet_verify_gb300 as gdn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


# activation rows -> stages of the ring: 32: 5, 96 .. 160: 3
@pytest.mark.parametrize("M", [16, 32, 96, 128, 144, 160])
def test_out_projection_over_a_long_k(M):
    g = torch.Generator(device="cuda").manual_seed(M)
    E, heads, d = 2560, 48, 128
    K = heads * d
    dims = gdn.make_dims(M // 16, 16, heads, d, d, 16)
    w_in = torch.zeros(8, dtype=torch.bfloat16, device="cuda")          # not read by this projection
    sets = []
    for _ in range(6):                                                  # 190 MB of weights: never all in L2
        w = (torch.randn((E, K), generator=g, device="cuda") * K ** -0.5).to(torch.bfloat16)
        x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
        ref = x.double() @ w.double().T
        # fp32 sums of K products (K 2^-24 of their magnitudes, taken twice), then one bf16 rounding
        err = K * 2.0 ** -23 * (x.double().abs() @ w.double().abs().T)
        sets.append((w, x, ref, 2.0 ** -8 * (ref.abs() + err) + err, gdn.proj_weights(E, w_in, w)))
    y = torch.empty((len(sets), M, E), dtype=torch.bfloat16, device="cuda")
    before = [torch.empty((M, E), dtype=torch.bfloat16, device="cuda") for _ in sets]
    for _ in range(100):
        for i, s in enumerate(sets):
            gdn.gdn_project_out(dims, s[4], s[1], before[i], None, 0)
    for i, s in enumerate(sets):
        gdn.gdn_project_out(dims, s[4], s[1], y[i], None, 0)
    torch.cuda.synchronize()
    for i, (_, _, ref, bound, _) in enumerate(sets):
        assert torch.equal(before[i], y[i])                        # every launch gives the same bits
        assert ((y[i].double() - ref).abs() <= bound).all()
