"""A row of equal values comes out as that value: the weights that values are multiplied with are those that are summed."""
import math

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


SIZES = [dict(T=1, H=8, Hk=2, D=128, page=16, past=[2, 3, 40, 700, 3000]),
         dict(T=5, H=6, Hk=1, D=256, page=64, past=[2, 500, 9000]),
         dict(T=2, H=8, Hk=2, D=64, page=16, past=[1, 900]),
         dict(T=40, H=8, Hk=2, D=64, page=16, past=[0, 500]),
         dict(T=40, H=4, Hk=1, D=256, page=16, past=[3, 300], window=60, n_sink=2),
         dict(T=16, H=24, Hk=4, D=128, page=32, past=[5, 1000], tree=True)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("alike", [False, True])
@pytest.mark.parametrize("sizes", SIZES)
def test_equal_values(sizes, alike, dtype):
    """A column's value c at every position, every number of a bf16's 7 bits among them.  sum w c / sum w is off by the sums'
    roundings alone, (n + 64) 2^-23 of c as in the other tests.  In bf16 that is far below half a step, so c itself has to
    come out.  alike: of all weights but that of position 0, which is 1, each is 0.5019 and rounded down to 0.5 in bf16."""
    c = Case(dtype=dtype, scale=-math.log(0.5019) if alike else None, **sizes)
    r = Run(c)
    columns = 1 + (torch.arange(c.Hk * c.D) * 37 % 128).view(c.Hk, c.D) / 128
    for s in range(c.B):
        for i in range(-(-(c.past[s] + c.n(s)) // c.page)):
            c.rows(r.vp)[int(c.table[s, i])] = columns.to(c.dtype)[:, None]
            if alike:                                       # q.k is 0 at position 0, else -1
                c.rows(r.kp)[int(c.table[s, i])] = 0
                c.rows(r.kp)[int(c.table[s, i]), :, (1 if i == 0 else 0):, 0] = -1
    if alike:
        r.q[:] = 0
        r.q[..., 0] = 1
    r.gpu.update(k=r.kp.cuda(), v=r.vp.cuda(), q=r.q.cuda())
    r.call()
    got = r.got()
    assert int(r.status.item()) == 0
    for s in range(c.B):
        want = columns.to(c.dtype).repeat_interleave(c.H // c.Hk, 0).expand(c.n(s), c.H, c.D)
        if dtype == "bf16":
            assert torch.equal(got[s, :c.n(s)], want), s
        else:
            n = c.past[s] + c.n(s)
            off = (got[s, :c.n(s)].double() - want.double()).abs() - (n + 64) * 2.0 ** -23 * want.abs()
            assert float(off.max()) <= 0, s
