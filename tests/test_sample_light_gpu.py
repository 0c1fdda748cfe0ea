"""gdn_sample where tokens are light: weights count in multiples of 2^-44 of the top one, so a token of less than half
of that is never drawn, and the sums are those of the rounded weights."""
import numpy as np
import pytest
import torch

import gated_deltanet_verify_gb300 as gdn
from tests.test_sample_gpu import run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


# one row in a cluster, a few, and one CTA a row
@pytest.mark.parametrize("rows,V", [(1, 40000), (3, 5000), (40, 9001), (200, 1500)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kw", [{}, dict(top_p=0.9999), dict(top_k=7), dict(top_k=1200), dict(min_p=1e-9)])
def test_the_first_draw_is_the_first_token_that_has_weight(kw, dtype, rows, V):
    # u = 0: the first kept token in index order with at least half a unit.  32 and 745 nats below the top a token has
    # none (2^-46.2 of the top weight, and nothing in 64 bits either), and neither has the type's lowest value; 26 nats
    # below it has 89 units
    logits = torch.full((rows, V), torch.finfo(dtype).min, dtype=dtype, device="cuda")
    logits[:, 1:300] = -32.0
    logits[:, 300:310] = -745.0
    logits[:, 900] = -26.0
    logits[:, 1100:1105] = -0.5
    logits[:, 1400] = 0.0
    one = {k: [v] * rows for k, v in kw.items()}
    tokens, lp = run(logits, torch.zeros(rows, 1, device="cuda"), temp=[1.0] * rows, **one)
    want = 900 if not kw or kw.get("top_k") == 1200 or kw.get("top_k") == 7 else 1100
    assert (tokens == want).all(), (want, tokens.unique())
    # top-p 0.9999 and min-p keep the six heavy tokens; e^-26 and less change the sum's logarithm by under 1e-8
    ref = (-26.0 if want == 900 else -0.5) - np.log(1 + 5 * np.exp(-0.5))
    assert (lp.double() - ref).abs().max() <= 4 * 2.0 ** -24 * abs(ref) + V * 2.0 ** -44 + 1e-8


@pytest.mark.parametrize("rows", [1, 200])
@pytest.mark.parametrize("nats", [31.0, 31.3])
def test_sums_are_those_of_the_rounded_weights(nats, rows):
    # 20000 tokens of 0.60 units count one each, of 0.45 none: e^-31 2^44 = 0.6056, e^-31.3 2^44 = 0.4487, the top
    # weight's own reference at most 2 * 2^-10 octaves above it (0.14 %)
    V = 20001
    logits = torch.full((rows, V), -nats, dtype=torch.float32, device="cuda")
    logits[:, V - 1] = 0.0
    unit = np.exp(-nats) * 2.0 ** 44
    units = round(unit)
    assert abs(unit - 0.5) > 0.05 * unit
    # behind the 3rd unit of a sum of 2^44 and up to 20000 of them; the top token lies behind all of them
    u = torch.full((rows, 1), 3.5 * 2.0 ** -44, dtype=torch.float32, device="cuda")
    tokens, lp = run(logits, u, temp=[1.0] * rows)
    assert (tokens == (3 if units else V - 1)).all(), tokens.unique()
    tokens, lp = run(logits, torch.full((rows, 1), 0.5, device="cuda"), temp=[1.0] * rows)
    assert (tokens == V - 1).all()
    assert lp.abs().max() <= 2 * V * 2.0 ** -44          # ln(1 + 20000 units)
