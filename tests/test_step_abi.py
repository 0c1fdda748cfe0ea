"""Host validation of the adapters, sampling and acceptance calls (no GPU needed), and the plain forms the GPU tests
compare with, pinned on hand-worked cases."""
import ctypes
import math

import numpy as np
import pytest

import gated_deltanet_verify_gb300 as gdn
from tests.step_ref import accept_row, accept_tree_row, lora, sample_row

A = 0x10000          # fake, aligned device address: never dereferenced (validation fails first)
ref = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build_library()
    return gdn.lib()


def dims(**kw):
    base = dict(n_slots=2, n_qk_heads=2, n_v_heads=8, d_k=32, d_v=32, n_tokens=4, act_dtype=gdn.GDN_BF16)
    base.update(kw)
    return gdn.make_dims(**base)


def test_sample_validation(lib):
    def call(d=None, logits=A, u=A, tokens=A, lp=None, params=(None,) * 4, **kw):
        base = dict(n_slots=2, n_tokens=3, vocab=100, ld=100, dtype=gdn.GDN_F32)
        base.update(kw)
        return lib.gdn_sample(ref(d or gdn.make_sample_dims(**base)), ref(gdn.sample_params(*params)), logits, u, tokens, lp,
                              None, None)

    for kw in (dict(vocab=0), dict(vocab=524289, ld=600000), dict(ld=99), dict(n_slots=0), dict(n_tokens=0),
               dict(n_slots=1 << 14, n_tokens=1 << 14)):
        assert call(**kw) == gdn.GDN_ERR_SHAPE, kw
    assert call(dtype=5) == gdn.GDN_ERR_DTYPE
    assert call(logits=None) == call(u=None) == call(tokens=None) == gdn.GDN_ERR_ARG
    assert call(logits=A + 4) == call(u=A + 4) == call(tokens=A + 8) == call(lp=A + 4) == gdn.GDN_ERR_ALIGN
    for i in range(4):
        assert call(params=[A + 4 if j == i else None for j in range(4)]) == gdn.GDN_ERR_ALIGN
    assert lib.gdn_sample(None, ref(gdn.sample_params()), A, A, A, None, None, None) == gdn.GDN_ERR_ARG
    assert gdn.gdn_last_error()


def test_accept_validation(lib):
    def chain(d=None, draft=A, tokens=A, length=None, trim=A, nxt=None, emit=None):
        return lib.gdn_accept(ref(d or dims()), draft, tokens, length, trim, nxt, emit, None, None)

    assert chain(d=dims(n_tokens=65)) == chain(d=dims(n_tokens=0)) == gdn.GDN_ERR_SHAPE
    assert chain(draft=None) == chain(tokens=None) == chain(trim=None) == gdn.GDN_ERR_ARG
    for k in ("draft", "tokens", "length", "trim", "nxt", "emit"):
        assert chain(**{k: A + 4}) == gdn.GDN_ERR_ALIGN, k
    assert lib.gdn_accept_tree(ref(dims()), None, A, A, None, A, None, None, None, None, None) == gdn.GDN_ERR_ARG
    assert lib.gdn_accept_tree(ref(dims()), A + 4, A, A, None, A, None, None, None, None, None) == gdn.GDN_ERR_ALIGN
    assert lib.gdn_accept_tree(ref(dims()), A, A, A, None, A, None, None, A + 4, None, None) == gdn.GDN_ERR_ALIGN


def test_lora_validation(lib):
    w = gdn.ProjWeights(64, A, A)
    good = dict(n_adapters=2, rank=16, a=A, b=A, scale=None)
    need = gdn.gdn_lora_workspace_bytes(dims(), 16)
    assert need >= 8 * 16 * 4 and need % 256 == 0
    assert gdn.gdn_lora_workspace_bytes(dims(), 12) == gdn.gdn_lora_workspace_bytes(dims(), 136) == 0

    for f in (lib.gdn_project_in_lora, lib.gdn_project_out_lora):
        def call(d=None, ww=w, ids=A, x=A, y=A, ws=A, n=need, **kw):
            return f(ref(d or dims()), ref(ww), ref(gdn.lora(**{**good, **kw})), ids, x, y, ws, n, None, None)

        assert call(rank=12) == call(rank=0) == call(rank=136) == call(n_adapters=0) == gdn.GDN_ERR_SHAPE
        assert call(a=None) == call(b=None) == call(ids=None) == call(x=None) == call(y=None) == gdn.GDN_ERR_ARG
        assert call(a=A + 2) == call(b=A + 2) == call(scale=A + 4) == call(ids=A + 4) == call(x=A + 2) == gdn.GDN_ERR_ALIGN
        assert call(ws=None) == call(n=need - 1) == gdn.GDN_ERR_WORKSPACE
        assert call(ws=A + 16) == gdn.GDN_ERR_ALIGN
        assert call(d=dims(act_dtype=gdn.GDN_F32)) == gdn.GDN_ERR_DTYPE
        assert call(ww=gdn.ProjWeights(60, A, A)) == gdn.GDN_ERR_SHAPE
        assert f(ref(dims()), ref(w), None, A, A, A, A, need, None, None) == gdn.GDN_ERR_ARG

    params = gdn.layer_params(A, A, A, A)
    lo = gdn.lora(**good)
    size = gdn.gdn_layer_lora_workspace_bytes(dims(), 64, 16)
    assert size >= gdn.gdn_layer_workspace_bytes(dims(), 64) + need

    def layer(i=lo, o=lo, ids=A, ws=A, n=size):
        p = lambda v: None if v is None else ref(v)  # noqa: E731
        return lib.gdn_layer_verify_lora(ref(dims()), ref(params), ref(w), p(i), p(o), ids, A, A, A, None, None, A, ws, n, None,
                                         None)

    assert layer(i=None, o=None) == gdn.GDN_ERR_ARG
    assert layer(ids=None) == gdn.GDN_ERR_ARG
    assert layer(n=size - 1) == layer(ws=None) == gdn.GDN_ERR_WORKSPACE
    assert layer(ws=A + 16) == gdn.GDN_ERR_ALIGN
    assert layer(o=gdn.lora(**{**good, "rank": 20})) == gdn.GDN_ERR_SHAPE


def test_plain_sampling_on_worked_cases():
    l = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
    # running sums in index order: .1 .5 .7 1
    assert [sample_row(l, u=u)[0] for u in (0.0, 0.09, 0.11, 0.49, 0.51, 0.69, 0.71, 0.99)] == [0, 0, 1, 1, 2, 2, 3, 3]
    # the two most likely are 1 and 3: 4/7 and 3/7
    assert [sample_row(l, top_k=2, u=u)[0] for u in (0.0, 0.57, 0.58)] == [1, 1, 3]
    assert [sample_row(l, top_p=0.6, u=u)[0] for u in (0.0, 0.57, 0.58)] == [1, 1, 3]
    assert [sample_row(l, top_p=0.75, u=u)[0] for u in (0.44, 0.45, 0.66, 0.67)] == [1, 2, 2, 3]      # 1, 3 and 2
    assert [sample_row(l, min_p=0.6, u=u)[0] for u in (0.57, 0.58)] == [1, 3]                         # .3 / .4 stays, .2 / .4 goes
    # top-p over what top-k left: of 4/7 and 3/7 the first reaches one half
    assert sample_row(l, top_k=2, top_p=0.5, u=0.99)[0] == 1
    assert sample_row(l, temp=0)[0] == 1 and sample_row(np.array([1.0, 2, 2]), temp=0)[0] == 1
    assert math.isclose(sample_row(l, top_k=2, u=0.9)[1], math.log(3 / 7))
    assert sample_row(np.array([-np.inf, np.nan])) == (-1, -math.inf)
    assert sample_row(np.array([1.0, 1, 1, 1]), top_k=3, u=0.99)[0] == 2


def test_plain_acceptance_on_worked_cases():
    assert accept_row([9, 1, 2, 3], [1, 2, 7, 8], 4, 4) == (1, 7, [1, 2, 7, -1])
    assert accept_row([9, 1, 2, 3], [1, 2, 7, 8], 2, 4) == (2, 2, [1, 2, -1, -1])
    assert accept_row([9, 0, 0, 0], [1, 2, 7, 8], 4, 4) == (3, 1, [1, -1, -1, -1])
    assert accept_row([9, 1, 2, 7], [1, 2, 7, 8], 4, 4) == (0, 8, [1, 2, 7, 8])
    parent, draft, tokens = [-1, 0, 0, 1, 2, 2], [9, 5, 6, 1, 1, 2], [6, 0, 2, 0, 0, 4]
    assert accept_tree_row(parent, draft, tokens, 6, 6) == (5, 4, [6, 2, 4, -1, -1, -1], [0, 2, 5, -1, -1, -1])
    assert accept_tree_row(parent, draft, tokens, 5, 6)[0] == 2
    assert accept_tree_row(parent, draft, tokens, 0, 6)[0] == -1


def test_plain_adapters_on_a_worked_case():
    x, w = np.array([[1.0, 2], [3, 4]]), np.array([[1.0, 0], [0, 1], [1, 1]])
    a, b = np.array([[[1.0, 1]]]), np.array([[[1.0], [0], [2]]])
    y, _ = lora(x, w, a, b, [0.5], [-1, 0], 1)
    assert y.tolist() == [[1, 2, 3], [6.5, 4, 14]]
