"""gdn_attend at the limits of its arguments: the widest windows, scales of nothing and next to nothing, the last positions."""
import pytest
import torch

import gated_deltanet_verify_gb300 as gdn
from tests.attn_ref import Case, attend_bound, attend_ref
from tests.test_attend_gpu import Run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 100, 2 ** 30, 2 ** 30 + 1])
@pytest.mark.parametrize("n_sink", [0, 3])
@pytest.mark.parametrize("sizes", [dict(T=1, H=8, Hk=2, D=128, page=16, past=[10, 0, 127, 500]),
                                   dict(T=20, H=8, Hk=2, D=64, page=16, past=[10, 0, 300]),
                                   dict(T=16, H=4, Hk=1, D=256, page=16, past=[10, 0, 300], tree=True)])
def test_windows_wider_than_any_cache(sizes, n_sink, window, dtype):
    r = Run(Case(dtype=dtype, window=window, n_sink=n_sink, **sizes))
    r.call()
    r.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -112, -(2.0 ** -114), 2.0 ** -140])
@pytest.mark.parametrize("rows", [1, 12])
def test_large_scores_under_a_small_scale(rows, scale, dtype):
    """Queries and keys of 2^53: scores of some 2^109, which a scale brings to some 10, to 1 or to nothing (2^-140 is below
    the smallest normal number)."""
    r = Run(Case(dtype=dtype, T=rows, H=8, Hk=2, D=64, page=16, past=[300, 5], scale=scale))
    big = 2.0 ** 53
    r.q, r.ks = r.q * big, [k * big for k in r.ks]
    r.gpu["q"], r.gpu["k"] = r.q.cuda(), r.gpu["k"] * big
    r.call()
    r.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("T,H", [(1, 2), (3, 4), (40, 8)])
def test_at_the_last_position(T, H, tree, dtype):
    """A window and first tokens at the end of the longest cache, 2^30 positions: only the pages that hold something seen are
    there."""
    D, page, window, n_sink = 64, 256, 300, 5
    past, max_pages = 2 ** 30 - T, 2 ** 30 // page
    c = Case(dtype=dtype, T=T, H=H, Hk=1, D=D, page=page, past=[0], length=[0], seed=T)
    g = c.g
    low = (past - window) // page
    pages = [0] + list(range(low, max_pages))
    pool = {n: torch.randn((len(pages) + 1, 1, page, D), generator=g).to(c.dtype) for n in "kv"}
    table = torch.full((1, max_pages), -1, dtype=torch.int32, device="cuda")
    for i, p in enumerate(pages):
        table[0, p] = i + 1
    q = (torch.randn((1, T, H, D), generator=g) * 1.5).to(c.dtype)
    parent = c.parents() if tree else None
    dims = gdn.make_attn_dims(1, T, H, 1, D, page, len(pages) + 1, max_pages,
                              dtype=gdn.GDN_F32 if dtype == "f32" else gdn.GDN_BF16)
    size = gdn.gdn_attend_workspace_bytes(dims)
    space = torch.empty(size, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.zeros((1, T, H, D), dtype=c.dtype, device="cuda")
    cache = gdn.kv_cache(pool["k"].cuda(), pool["v"].cuda(), table, torch.tensor([past], dtype=torch.int32, device="cuda"))
    gdn.gdn_attend(dims, cache, gdn.attn_params(D ** -0.5, window, n_sink), q.cuda(), out, space, size,
                   d_parent=parent.cuda() if tree else None, d_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    # the same among the positions that are there: from the first one that any token sees on they are numbered 5, 6, ...
    first = past - window + 1
    there = list(range(n_sink)) + list(range(first, past + T))
    at = torch.tensor([(pages.index(p // page) + 1) * page + p % page for p in there])
    keys, values = (pool[n].view(-1, D)[at].unsqueeze(1) for n in "kv")
    near = Case(dtype=dtype, T=T, H=H, Hk=1, D=D, page=page, past=[len(there) - T], tree=tree, window=window)
    near.n_sink = n_sink
    want, mass, reach = attend_ref(near, q, [keys], [values], parent)[0]
    off = (out[0].cpu().double() - want).abs() - attend_bound(near, 0, want, mass, reach)
    assert float(off.max()) <= 0
