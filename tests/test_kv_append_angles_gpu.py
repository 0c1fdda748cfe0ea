"""The append's angles at far positions and for all frequencies, against angles from 100 decimal digits."""
import decimal
import math

import pytest
import torch

import gated_deltanet_verify_gb300 as gdn

pytestmark = pytest.mark.gpu

PI = decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798214808651")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def turns(freq, position):
    """freq * position / 2 pi less its whole turns; freq is an fp32 number, taken exactly."""
    with decimal.localcontext() as ctx:
        ctx.prec = 100
        x = decimal.Decimal(freq) * position / (2 * PI)
        return float(x - x.to_integral_value())


# frequencies of models, and others: negative, large, tiny, beside multiples of a turn
FREQ = [1.0, -1.0, 0.5, 1e-3, 1e-7, 1e-30, 2 * math.pi, math.pi, 10.0, 1000.0, -777.7, 1e6, 2.0 ** 20, 3.1e9, 2.0 ** 40, 0.0]


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("past", [0, 1000, 2 ** 20 - 2, 2 ** 24 + 1, 2 ** 30 - 3])
def test_angles(past, adjacent):
    """A unit vector along each pair's first number is turned to (cos, sin): off by 2^-24 of a turn and 2^-22 for cos and
    sin at most."""
    D, T, page = 64, 3, 256
    freq = torch.tensor(FREQ, dtype=torch.float32)
    half = len(FREQ)
    max_pages = 2 ** 30 // page
    table = torch.full((1, max_pages), -1, dtype=torch.int32, device="cuda")
    first, last = past // page, (past + T - 1) // page
    table[0, first], table[0, last] = 0, last - first
    k = torch.zeros((2, 1, page, D), device="cuda")
    v = torch.zeros_like(k)
    dims = gdn.make_attn_dims(1, T, 1, 1, D, page, 2, max_pages, dtype=gdn.GDN_F32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = torch.zeros((1, T, D), device="cuda")
    at = [(2 * i, 2 * i + 1) if adjacent else (i, i + half) for i in range(half)]
    for i, _ in at:
        x[..., i] = 1.0
    q = torch.zeros((1, T, 1, D), device="cuda")
    cache = gdn.kv_cache(k, v, table, torch.tensor([past], dtype=torch.int32, device="cuda"))
    gdn.gdn_kv_append(dims, cache, gdn.qk_params(2 * half, freq.cuda(), adjacent=adjacent), x, x, x, D, D, D, q, d_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    bound = 2 * math.pi * 2.0 ** -24 + 2.0 ** -22
    for t in range(T):
        p = past + t
        for y in (q[0, t, 0], k[p // page - first, 0, p % page]):
            y = y.tolist()
            for (i, j), f in zip(at, freq.tolist()):
                angle = 2 * math.pi * turns(f, p)
                assert abs(y[i] - math.cos(angle)) <= bound and abs(y[j] - math.sin(angle)) <= bound, (f, p)
