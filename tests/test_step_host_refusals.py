"""gdn_verify_step_host refuses what its verify and its rollback would refuse before it copies anything (on a machine
without a GPU a copy that came first would show as GDN_ERR_LAUNCH)."""
import ctypes

import pytest

import gated_deltanet_verify_gb300 as gdn

A = 0x10000          # fake, aligned device address: never dereferenced
ref = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build_library()
    return gdn.lib()


@pytest.mark.parametrize("rollback_first", [0, 1])
@pytest.mark.parametrize("what,value,code", [
    ("state", None, gdn.GDN_ERR_ARG), ("state", A + 4, gdn.GDN_ERR_ALIGN), ("conv_state", None, gdn.GDN_ERR_ARG),
    ("cap_state", None, gdn.GDN_ERR_NO_CAPTURE), ("cap_conv", None, gdn.GDN_ERR_NO_CAPTURE),
    ("cap_state", A + 8, gdn.GDN_ERR_ALIGN), ("cap_conv", A + 4, gdn.GDN_ERR_ALIGN), ("params", None, gdn.GDN_ERR_ARG),
    ("dims", dict(n_tokens=65), gdn.GDN_ERR_SHAPE), ("dims", dict(d_k=48), gdn.GDN_ERR_SHAPE),
    ("dims", dict(n_slots=65536), gdn.GDN_ERR_SHAPE),
])
def test_every_check_comes_before_the_copy(lib, rollback_first, what, value, code):
    kw = dict(n_slots=2, n_qk_heads=2, n_v_heads=8, d_k=32, d_v=32, n_tokens=4, act_dtype=gdn.GDN_BF16)
    if what == "dims":
        kw.update(value)
    b = {**dict(state=A, conv_state=A, cap_state=A, cap_conv=A), **({what: value} if what.startswith(("s", "c")) else {})}
    p = gdn.layer_params(value, A, A, A) if what == "params" else gdn.layer_params(A, A, A, A)
    got = lib.gdn_verify_step_host(ref(gdn.make_dims(**kw)), ref(p), rollback_first, A, A, A, 1 << 60, b["state"],
                                   b["conv_state"], b["cap_state"], b["cap_conv"], None, None)
    assert got == code, gdn.gdn_last_error()
