"""Projections of more rows or columns than a launch can hold are refused by their size, before any arithmetic on it
could overflow (no GPU needed: a call that came as far as a launch would answer GDN_ERR_LAUNCH)."""
import ctypes

import pytest

import gated_deltanet_verify_gb300 as gdn

A = 0x10000          # fake, aligned device address: never dereferenced
ref = ctypes.byref
ROWS = 65535 * 256


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build_library()
    return gdn.lib()


def dims(**kw):
    return gdn.make_dims(**{**dict(n_slots=2, n_qk_heads=2, n_v_heads=8, d_k=32, d_v=32, n_tokens=4,
                                   act_dtype=gdn.GDN_BF16), **kw})


# 2^23 tiles of columns times 2^22 blocks of rows is 0 in 32 bits
@pytest.mark.parametrize("kw,embd", [
    (dict(n_slots=ROWS + 1, n_tokens=1), 64), (dict(n_slots=1 << 15, n_tokens=1 << 15), 64),
    (dict(n_slots=1 << 30, n_tokens=1, n_v_heads=8, n_qk_heads=8, d_v=(1 << 26) - 64), 64),
    (dict(n_slots=1 << 30, n_tokens=1), 1 << 30), (dict(n_slots=1 << 16, n_tokens=1 << 16), 64),
    (dict(), (1 << 30) + 8), (dict(), (1 << 31) - 8),
])
def test_sizes_that_no_launch_holds(lib, kw, embd):
    d, w = dims(**kw), gdn.ProjWeights(embd, A, A)
    lo = gdn.lora(2, 16, A, A)
    assert lib.gdn_project_in(ref(d), ref(w), A, A, None, 0, None) == gdn.GDN_ERR_SHAPE
    assert lib.gdn_project_out(ref(d), ref(w), A, A, None, 0, None) == gdn.GDN_ERR_SHAPE
    for f in (lib.gdn_project_in_lora, lib.gdn_project_out_lora):
        assert f(ref(d), ref(w), ref(lo), A, A, A, A, 1 << 62, None, None) == gdn.GDN_ERR_SHAPE


def test_the_adapters_workspace_is_0_where_the_call_is_refused(lib):
    for kw in (dict(n_slots=ROWS + 1, n_tokens=1), dict(n_slots=1 << 30, n_tokens=1 << 30),
               dict(n_slots=(1 << 31) - 1, n_tokens=(1 << 31) - 1)):
        assert gdn.gdn_lora_workspace_bytes(dims(**kw), 128) == 0
        assert gdn.gdn_layer_lora_workspace_bytes(dims(**kw), 64, 128) == 0
    assert gdn.gdn_lora_workspace_bytes(dims(n_slots=ROWS, n_tokens=1), 128) >= ROWS * 128 * 4
