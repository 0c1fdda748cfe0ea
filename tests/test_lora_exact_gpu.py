"""h = scale A x of an adapter is carried to the second product in all the bits of its fp32 sum: on whole numbers, where
every sum is exact, rank columns that cancel leave exactly what they differ by."""
import pytest
import torch

import gated_deltanet_verify_gb300 as gdn
from tests.test_lora_gpu import Case, shape_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("side", ["in", "out"])
@pytest.mark.parametrize("rank", [8, 16, 32, 64, 72, 128])
@pytest.mark.parametrize("B,T", [(1, 1), (3, 5), (2, 16), (9, 16), (20, 15)])
def test_what_cancels_leaves_the_difference(side, rank, B, T):
    c = Case(shape_of(n_slots=B, n_tokens=T), side, 3, rank, [i % 4 - 1 if B > 1 else 2 for i in range(B)], seed=rank, scale=False)
    g = torch.Generator(device="cuda").manual_seed(rank + T)
    digit = lambda *s: torch.randint(-127, 128, s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    c.w.zero_()
    c.x.zero_()
    c.a.zero_()
    # x = sign (1, 2^7, 2^14), so h is a whole number of up to 21 bits whose digits are A's; the rank columns come in
    # pairs that differ in the lowest digit, and B takes one from the other
    sign = torch.randint(0, 2, (c.M,), generator=g, device="cuda") * 2 - 1
    for k in range(3):
        c.x[:, k] = sign * 2.0 ** (7 * k)
        c.a[:, 0::2, k] = digit(3, rank // 2)
        c.a[:, 1::2, k] = c.a[:, 0::2, k] if k else digit(3, rank // 2)
    c.b[:, :, 0::2] = torch.randint(-1, 2, (3, c.N, rank // 2), generator=g, device="cuda").to(torch.bfloat16)
    c.b[:, :, 1::2] = -c.b[:, :, 0::2]
    y = c.run()
    want = torch.zeros((c.M, c.N), dtype=torch.float64, device="cuda")
    for s, i in enumerate(c.ids.tolist()):
        if i >= 0:
            rows = slice(s * T, (s + 1) * T)
            want[rows] = c.x[rows].double() @ c.a[i].double().T @ c.b[i].double().T
    assert want.abs().max() > 100
    # at most 254 * 64 < 2^14: exact in fp32, so one rounding to bf16 is all that is left
    assert torch.equal(y, want.float().to(torch.bfloat16))


def test_a_large_h_stays_finite():
    # 2^127 (2 - 2^-9), between bf16's largest number and 2^128, is a number in fp32 but rounds to infinity in bf16
    c = Case(shape_of(n_slots=1, n_tokens=3), "in", 1, 8, [0], scale=False)
    for t in (c.w, c.x, c.a, c.b):
        t.zero_()
    c.x[:, 0], c.x[:, 1] = 2.0 ** 64, 2.0 ** 55
    c.a[:, :, 0], c.a[:, :, 1] = 2.0 ** 63 * (2 - 2.0 ** -7), 2.0 ** 64 * 1.5
    c.b[:, :, 0] = 2.0 ** -60
    h = 2.0 ** 127 * (2 - 2.0 ** -7) + 2.0 ** 119 * 1.5
    assert h < 2.0 ** 128 * (1 - 2.0 ** -24)
    y = c.run()
    assert (y.double() == float(torch.tensor(h * 2.0 ** -60, dtype=torch.float32).to(torch.bfloat16))).all(), y
