"""gdn_sample against the plain 64-bit form: filters, ties, masks, strides, types, sizes, refusals."""
import numpy as np
import pytest
import torch

import gated_deltanet_verify_gb300 as gdn
from tests.step_ref import sample_row

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


F = lambda v: torch.tensor(v, dtype=torch.float32, device="cuda")  # noqa: E731
I = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731


def run(logits, u, temp=None, top_k=None, top_p=None, min_p=None, T=1, vocab=None, status=None, **kw):
    """logits [B*T][ld] on the device; parameters as lists per slot or None."""
    rows, ld = logits.shape
    B = rows // T
    t = [None if v is None else f(v) for f, v in ((F, temp), (I, top_k), (F, top_p), (F, min_p))]
    tokens = torch.full((B, T), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((B, T), 7.0, dtype=torch.float32, device="cuda")
    dims = gdn.make_sample_dims(B, T, ld if vocab is None else vocab, ld=ld,
                                dtype=gdn.GDN_BF16 if logits.dtype == torch.bfloat16 else gdn.GDN_F32)
    gdn.gdn_sample(dims, gdn.sample_params(*t), logits, u, tokens, lp, status, **kw)
    return tokens, lp


def check(logits, u, temp=None, top_k=None, top_p=None, min_p=None, T=1, vocab=None):
    tokens, lp = run(logits, u, temp, top_k, top_p, min_p, T, vocab)
    torch.cuda.synchronize()
    V = logits.shape[1] if vocab is None else vocab
    host, uh = logits[:, :V].double().cpu().numpy(), u.double().cpu().numpy().reshape(-1)
    tok, lph = tokens.cpu().numpy().reshape(-1), lp.double().cpu().numpy().reshape(-1)
    f32 = lambda v: float(np.float32(v))  # noqa: E731
    for i in range(host.shape[0]):
        s = i // T
        ref = sample_row(host[i], 1.0 if temp is None else f32(temp[s]), 0 if top_k is None else top_k[s],
                         1.0 if top_p is None else f32(top_p[s]), 0.0 if min_p is None else f32(min_p[s]), uh[i])
        assert tok[i] == ref[0], (i, tok[i], ref)
        if ref[0] < 0:
            assert lph[i] == -np.inf
        else:
            # x - ln(sum), both terms <= 0: x is a rounded quotient of a rounded difference (2 units of 2^-24 of it), the
            # logarithm is within 1 ulp (2 units) of a rounded argument (1 unit), their difference is rounded (1 unit): 4
            # units of the whole at most; the sum itself is within 2^-44 of the top weight a token, and 2^-34 of those
            # tokens' weights that are below 2^-4 of the top one: less than 2^-34 of ln(sum / top), which the token pays too
            assert abs(lph[i] - ref[1]) <= 4 * 2.0 ** -24 * abs(ref[1]) + V * 2.0 ** -44 + 1e-12, (i, lph[i], ref)


def logits_of(rows, V, dtype=torch.float32, seed=0, std=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((rows, V), generator=g, device="cuda") * std).to(dtype)


def uniforms(rows, T=1, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand((rows // T, T), generator=g, device="cuda")


FILTERS = {
    "none": {},
    "top_k": dict(top_k=[1, 3, 50, 0]),
    "top_p": dict(top_p=[0.1, 0.5, 0.9, 0.999]),
    "min_p": dict(min_p=[0.9, 0.3, 0.05, 1e-6]),
    "all": dict(top_k=[40, 40, 7, 100000], top_p=[0.9, 0.35, 0.95, 0.8], min_p=[0.02, 0.01, 0.2, 0.0]),
    "greedy_among": dict(temp=[0.0, 0.8, 0.0, 1.7], top_k=[0, 5, 3, 0]),
}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 31, 257, 1000, 4099, 32768, 50257])
@pytest.mark.parametrize("name", sorted(FILTERS))
def test_filters_and_sizes(name, V, dtype):
    kw = dict(FILTERS[name])
    kw.setdefault("temp", [0.7, 1.0, 1.3, 0.9])
    T = 3
    check(logits_of(4 * T, V, dtype, seed=V), uniforms(4 * T, T, seed=V + 1), T=T, **kw)


@pytest.mark.parametrize("V,dtype", [(200001, torch.float32), (200001, torch.bfloat16), (524288, torch.float32),
                                     (524288, torch.bfloat16)])
def test_large_vocabularies(V, dtype):
    check(logits_of(4, V, dtype, seed=5), uniforms(4, seed=6), temp=[1.0, 0.8, 1.1, 0.9], top_k=[0, 0, 60, 0],
          top_p=[1.0, 0.95, 0.9, 1.0], min_p=[0.0, 0.0, 0.0, 0.03])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("std,temp", [(1.0, 1.3), (0.05, 1.0), (4.0, 900.0), (2.0, 2.0 ** 20), (6.0, 0.02)])
def test_borders_among_many_tokens(std, temp, dtype):
    # nearly flat rows: thousands of tokens around the border, equal ones (bf16) or different ones
    l = logits_of(6, 150001, dtype, seed=40, std=std)
    check(l, uniforms(6, seed=41), temp=[temp] * 6, top_p=[0.3, 0.7, 0.95, 0.999, 1.0, 0.9],
          top_k=[0, 0, 0, 0, 40000, 100000])
    check(l, uniforms(6, seed=42), temp=[temp] * 6, top_k=[600, 3000, 20000, 75000, 150000, 1023])


@pytest.mark.parametrize("rows", [1, 3, 40, 80, 200])
def test_launch_shapes(rows):
    # from many CTAs a row to one; the first k tokens in one place, so that few threads hold them
    l = logits_of(rows, 30011, seed=50 + rows)
    l[:, 4000:4400] += 20.0
    check(l, uniforms(rows, seed=3), temp=[0.9] * rows, top_k=[(7 * i) % 390 + 1 for i in range(rows)],
          top_p=[1.0 if i % 2 else 0.9 for i in range(rows)])


@pytest.mark.parametrize("pad", [1, 3, 8, 61])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_row_strides_and_what_lies_between_rows(pad, dtype):
    # rows start on every alignment of the type; the columns behind a row hold values that would win
    V = 4097
    logits = logits_of(10, V + pad, dtype, seed=pad)
    logits[:, V:] = 1e30
    check(logits, uniforms(10, 2), top_p=[0.9] * 5, temp=[1.0] * 5, T=2, vocab=V)
    check(logits, uniforms(10, 2), temp=[0.0] * 5, T=2, vocab=V)


def test_ties_are_kept_by_index():
    # few distinct values: the border of every filter lies among equals
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.randint(0, 4, (24, 3001), generator=g, device="cuda").float()
    for dtype in (torch.float32, torch.bfloat16):
        l = logits.to(dtype)
        check(l, uniforms(24, 4), temp=[1.0] * 6, top_k=[1, 10, 700, 751, 1500, 2999], T=4)
        check(l, uniforms(24, 4), temp=[1.0] * 6, top_p=[0.013, 0.2, 0.61, 0.77, 0.93, 0.99], T=4)
        check(l, uniforms(24, 4), temp=[2.0] * 6, top_k=[900] * 6, top_p=[0.013, 0.2, 0.61, 0.77, 0.93, 0.99], T=4)
        check(l, uniforms(24, 4), temp=[0.0] * 6, T=4)
    flat = torch.full((6, 2000), 1.25, device="cuda")
    check(flat, uniforms(6), temp=[1.0] * 6, top_k=[0, 1, 77, 2000, 1999, 0], top_p=[1.0, 1.0, 1.0, 1.0, 0.3331, 0.7777])
    zero = torch.zeros((4, 500), device="cuda")
    zero[:, ::2] = -0.0            # -0 equals 0: the lower index first
    check(zero, uniforms(4), temp=[0.0, 1.0, 1.0, 1.0], top_k=[0, 1, 2, 251])


@pytest.mark.parametrize("base", [1e8, -1e30, 3e38])
def test_large_logits(base):
    # a place of the largest is wider than the differences that the temperature tells apart (but the last temperature)
    V = 20001
    g = torch.Generator(device="cuda").manual_seed(77)
    step = 2.0 ** (np.floor(np.log2(abs(base))) - 23)
    l = (torch.randint(0, 12, (8, V), generator=g, device="cuda").double() * step + base).float()
    l[6:] = base                                      # all equal, as in a row of an additive mask
    for temp in (1.0, min(4.0 * step, 2.0 ** 20)):
        check(l, uniforms(8, seed=12), temp=[temp] * 8, top_p=[0.2, 0.5, 0.9, 0.99, 1.0, 1.0, 0.4, 0.9],
              top_k=[0, 0, 0, 5000, 700, 0, 0, 3])


def test_many_infinite_logits():
    l = logits_of(6, 40003, seed=13)
    l[:, ::2] = float("inf")
    check(l, uniforms(6, seed=14), temp=[1.0] * 6, top_k=[1, 9000, 20001, 20002, 30000, 0],
          top_p=[1.0, 0.5, 0.9, 1.0, 0.3, 0.7], min_p=[0.0, 0.0, 0.5, 0.0, 0.0, 1.0])


def test_masks_infinities_and_lowest_values():
    V = 1537
    for dtype in (torch.float32, torch.bfloat16):
        low = torch.finfo(dtype).min
        l = logits_of(12, V, dtype, seed=9)
        l[0] = float("-inf")                          # nothing allowed
        l[1] = float("nan")
        l[2] = float("-inf"); l[2, 1400] = -30.0      # one token allowed
        l[3] = low                                    # the lowest value everywhere: all equal
        l[4] = low; l[4, 700:] = float("-inf")
        l[5, 5] = float("inf")                        # one certain token
        l[6, 5] = float("inf"); l[6, 1300] = float("inf")
        l[7, ::3] = float("nan")
        l[8, 1:] = low
        l[9] = torch.finfo(dtype).max; l[9, ::2] = low
        l[10, : V - 1] = float("-inf")                # the last token alone
        l[11, 1:] = float("nan"); l[11, 0] = low
        for kw in ({}, dict(top_k=[4] * 12), dict(top_p=[0.77] * 12), dict(min_p=[0.1] * 12),
                   dict(top_k=[6] * 12, top_p=[0.9] * 12, min_p=[0.02] * 12)):
            check(l, uniforms(12, seed=11), temp=[1.0] * 12, **kw)
        check(l, uniforms(12, seed=11), temp=[0.0] * 12)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    run(l, uniforms(12), status=status)
    assert int(status) == gdn.GDN_ERR_SAMPLE


@pytest.mark.parametrize("temp", [2.0 ** -20, 0.01, 30.0, 2.0 ** 20])
def test_extreme_temperatures(temp):
    check(logits_of(6, 5003, seed=2), uniforms(6, seed=8), temp=[temp] * 6, top_p=[1.0, 1.0, 0.9, 0.9, 0.5, 0.5],
          top_k=[0, 20, 0, 20, 0, 20])


def test_extreme_uniforms():
    # 0 draws the first kept token, the largest below 1 the last one of any mass
    l = logits_of(4, 3001, seed=4)
    u = torch.tensor([[0.0], [1 - 2.0 ** -24], [2.0 ** -149], [0.5]], device="cuda")
    check(l, u, temp=[1.0] * 4)
    check(l, u, temp=[1.0] * 4, top_k=[10] * 4)


@pytest.mark.parametrize("kw,u", [(dict(temp=[-1.0]), 0.5), (dict(temp=[float("nan")]), 0.5), (dict(temp=[2.0 ** -21]), 0.5),
                                  (dict(temp=[float("inf")]), 0.5), (dict(top_p=[0.0]), 0.5), (dict(top_p=[float("nan")]), 0.5),
                                  (dict(min_p=[1.5]), 0.5), (dict(min_p=[float("nan")]), 0.5), ({}, 1.0), ({}, -0.1),
                                  ({}, float("nan"))])
def test_refused_rows_are_reported(kw, u):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    tokens, lp = run(logits_of(1, 100), F([[u]]), status=status, **kw)
    assert int(tokens) == -1 and float(lp) == -np.inf and int(status) == gdn.GDN_ERR_SAMPLE


def test_rows_do_not_touch_each_other_and_outputs_stay_in_bounds():
    B, T, V = 3, 5, 2003
    l, u = logits_of(B * T, V, seed=12), uniforms(B * T, T)
    space = torch.full((B * T + 64,), 123, dtype=torch.int32, device="cuda")
    lps = torch.full((B * T + 64,), 5.0, device="cuda")
    dims, params = gdn.make_sample_dims(B, T, V), gdn.sample_params(top_p=F([0.9] * B))
    gdn.gdn_sample(dims, params, l, u, space, lps)
    torch.cuda.synchronize()
    assert (space[B * T:] == 123).all() and (lps[B * T:] == 5.0).all() and (space[:B * T] >= 0).all()
    one, _ = run(l[7:8].clone(), u.reshape(-1)[7:8].reshape(1, 1).clone(), top_p=[0.9])
    assert int(one) == int(space[7])
    again = torch.empty_like(space)
    gdn.gdn_sample(dims, params, l, u, again, None)
    assert torch.equal(again[:B * T], space[:B * T])


def test_many_rows():
    l, u = logits_of(700, 1031, torch.bfloat16, seed=21), uniforms(700, 7)
    check(l, u, temp=[0.5 + 0.01 * i for i in range(100)], top_k=[i % 40 for i in range(100)], T=7)


def test_rows_past_32_bit_offsets():
    ld = 1 << 28
    l = torch.empty((17, ld), dtype=torch.bfloat16, device="cuda")
    l[:, :1500] = logits_of(17, 1500, torch.bfloat16, seed=30)
    check(l, uniforms(17), vocab=1500, top_p=[0.95] * 17)


def test_graph_replay_and_another_stream():
    l, u = logits_of(16, 33001, seed=14), uniforms(16, 4)
    want, lp = run(l, u, temp=[0.9] * 4, top_p=[0.9] * 4, T=4)
    torch.cuda.synchronize()
    params = gdn.sample_params(F([0.9] * 4), None, F([0.9] * 4), None)
    dims = gdn.make_sample_dims(4, 4, 33001)
    tokens = torch.zeros((4, 4), dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gdn.gdn_sample(dims, params, l, u, tokens)
    side.synchronize()
    assert torch.equal(tokens, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gdn.gdn_sample(dims, params, l, u, tokens)
    l2 = logits_of(16, 33001, seed=15)
    l.copy_(l2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(tokens, run(l2, u, temp=[0.9] * 4, top_p=[0.9] * 4, T=4)[0])


def test_two_calls_at_once():
    # two streams, each with its own rows: no shared scratch
    a, b, u = logits_of(8, 90001, seed=1), logits_of(8, 90001, seed=2), uniforms(8)
    wa, wb = run(a, u, top_p=[0.9] * 8)[0], run(b, u, top_k=[50] * 8)[0]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        with torch.cuda.stream(s[0]):
            ga = run(a, u, top_p=[0.9] * 8)[0]
        with torch.cuda.stream(s[1]):
            gb = run(b, u, top_k=[50] * 8)[0]
        torch.cuda.synchronize()
        assert torch.equal(ga, wa) and torch.equal(gb, wb)
