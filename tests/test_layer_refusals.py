"""A layer call that is refused has enqueued nothing: every argument is checked before the first launch (on a machine
without a GPU a launch that came first would show as GDN_ERR_LAUNCH), and state, captures and workspace stay as they
were."""
import ctypes

import pytest
import torch

import gated_deltanet_verify_gb300 as gdn

A = 0x10000          # fake, aligned device address: never dereferenced
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


BUFFERS = dict(x=A, state=A, conv_state=A, cap_state=None, cap_conv=None, y=A)
LORA = dict(n_adapters=2, rank=16, a=A, b=A, scale=None)
WRONG = [("y", None, gdn.GDN_ERR_ARG), ("y", A + 8, gdn.GDN_ERR_ALIGN), ("x", None, gdn.GDN_ERR_ARG),
         ("x", A + 2, gdn.GDN_ERR_ALIGN), ("state", None, gdn.GDN_ERR_ARG), ("conv_state", A + 4, gdn.GDN_ERR_ALIGN),
         ("cap_state", A + 4, gdn.GDN_ERR_ALIGN), ("cap_conv", A + 8, gdn.GDN_ERR_ALIGN),
         ("params", None, gdn.GDN_ERR_ARG), ("params", A + 4, gdn.GDN_ERR_ALIGN),
         ("dims", dict(n_tokens=65), gdn.GDN_ERR_SHAPE), ("dims", dict(d_k=48), gdn.GDN_ERR_SHAPE),
         ("dims", dict(d_v=264), gdn.GDN_ERR_SHAPE), ("dims", dict(n_slots=65536, n_tokens=1), gdn.GDN_ERR_SHAPE),
         ("dims", dict(n_qk_heads=1, n_v_heads=24), gdn.GDN_ERR_SHAPE)]


@pytest.mark.parametrize("adapters", [None, "in", "out", "inout"])
@pytest.mark.parametrize("what,value,code", WRONG)
def test_every_check_comes_before_the_first_launch(lib, adapters, what, value, code):
    buf = dict(BUFFERS)
    d = dims(**value) if what == "dims" else dims()
    p = gdn.layer_params(value, A, A, A) if what == "params" else gdn.layer_params(A, A, A, A)
    if what in buf:
        buf[what] = value
    w, lo, tail = gdn.ProjWeights(64, A, A), gdn.lora(**LORA), (buf["y"], A, 1 << 40, None, None)
    b = [buf[k] for k in ("x", "state", "conv_state", "cap_state", "cap_conv")]
    if adapters is None:
        got = lib.gdn_layer_verify(ref(d), ref(p), ref(w), *b, *tail)
    else:
        got = lib.gdn_layer_verify_lora(ref(d), ref(p), ref(w), ref(lo) if "in" in adapters else None,
                                        ref(lo) if "out" in adapters else None, A, *b, *tail)
    assert got == code, gdn.gdn_last_error()


def test_too_many_adapters_of_the_output_side(lib):
    many = gdn.lora(**{**LORA, "n_adapters": 1 << 26})
    b = [BUFFERS[k] for k in ("x", "state", "conv_state", "cap_state", "cap_conv", "y")]
    for i in (None, gdn.lora(**LORA)):
        assert lib.gdn_layer_verify_lora(ref(dims()), ref(gdn.layer_params(A, A, A, A)), ref(gdn.ProjWeights(64, A, A)),
                                         i and ref(i), ref(many), A, *b, A, 1 << 40, None, None) == gdn.GDN_ERR_SHAPE
    for f in (lib.gdn_project_in_lora, lib.gdn_project_out_lora):
        assert f(ref(dims()), ref(gdn.ProjWeights(64, A, A)), ref(many), A, A, A, A, 1 << 40, None,
                 None) == gdn.GDN_ERR_SHAPE


@pytest.mark.gpu
@pytest.mark.parametrize("adapters", [False, True])
def test_a_refused_layer_call_changes_nothing(adapters):
    from tests.gpu_util import dims_of, params_of, upload
    from tests.test_lora_gpu import Case, shape_of
    from workloads.synth import make_inputs

    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    s = shape_of()
    i, o = Case(s, "in", 2, 16, [1, -1, 0], seed=1), Case(s, "out", 2, 16, [1, -1, 0], seed=2)
    x, d = upload(make_inputs(s)), dims_of(s)
    w = gdn.proj_weights(s.n_embd, i.w, o.w)
    size = gdn.gdn_layer_lora_workspace_bytes(d, s.n_embd, 16)
    space = torch.full((size,), 7, dtype=torch.uint8, device="cuda")
    y = torch.zeros(i.M * s.n_embd + 8, dtype=torch.bfloat16, device="cuda")
    state, conv = x["state"].clone(), x["conv_state"].clone()
    for bad in (None, y[1:]):
        with pytest.raises(gdn.GdnError):
            if adapters:
                gdn.gdn_layer_verify_lora(d, params_of(x), w, i.lora, o.lora, i.ids, i.x, x["state"], x["conv_state"], None,
                                          None, bad, space, size)
            else:
                gdn.gdn_layer_verify(d, params_of(x), w, i.x, x["state"], x["conv_state"], None, None, bad, space, size)
    torch.cuda.synchronize()
    assert torch.equal(x["state"], state) and torch.equal(x["conv_state"], conv)
    assert (space == 7).all() and (y == 0).all()
