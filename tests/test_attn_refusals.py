"""gdn_kv_append and gdn_attend refuse on the host what they cannot run (no GPU needed; nothing is dereferenced)."""
import ctypes
import math

import pytest

import gated_deltanet_verify_gb300 as gdn

A = 0x10000          # fake, 16-byte aligned device addresses


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build_library()


def dims(**kw):
    v = dict(n_slots=2, n_tokens=4, n_heads=8, n_kv_heads=2, d_head=64, page_tokens=16, n_pages=10, max_pages=5,
             dtype=gdn.GDN_BF16)
    v.update(kw)
    return gdn.make_attn_dims(**v)


def cache(**kw):
    v = dict(k=A, v=A, page_table=A, past=A)
    v.update(kw)
    return gdn.kv_cache(**v)


BAD_DIMS = [dict(n_slots=0), dict(n_tokens=0), dict(n_slots=2 ** 13, n_tokens=2 ** 12), dict(n_heads=7), dict(n_heads=0),
            dict(n_kv_heads=0), dict(n_heads=130, n_kv_heads=2), dict(n_heads=2 ** 17, n_kv_heads=2 ** 16),
            dict(n_slots=1, n_tokens=2 ** 23, n_heads=2 ** 10, n_kv_heads=2 ** 5), dict(d_head=96),
            dict(d_head=0), dict(page_tokens=4), dict(page_tokens=24), dict(page_tokens=512), dict(n_pages=0),
            dict(max_pages=0), dict(max_pages=2 ** 27), dict(page_stride=2 * 16 * 64 - 8), dict(page_stride=2 * 16 * 64 + 4),
            dict(page_stride=2 ** 38)]


def call_append(d=None, c=None, p=None, **kw):
    v = dict(q=A, k=A, v=A, ld_q=512, ld_k=128, ld_v=128, q_out=A + 16, d_length=None, d_parent=None, d_path=None)
    v.update(kw)
    p = gdn.qk_params(32, A, A, A) if p is None else p
    gdn.gdn_kv_append(d or dims(), c or cache(), p, v["q"], v["k"], v["v"], v["ld_q"], v["ld_k"], v["ld_v"], v["q_out"],
                      d_length=v["d_length"], d_parent=v["d_parent"], d_path=v["d_path"], stream=0)


def call_attend(d=None, c=None, p=None, **kw):
    d = d or dims()
    v = dict(q=A, out=A + 4096, workspace=A, ws_bytes=1 << 40, d_length=None, d_parent=None)
    v.update(kw)
    gdn.gdn_attend(d, c or cache(), p or gdn.attn_params(0.125), v["q"], v["out"], v["workspace"], v["ws_bytes"],
                   d_length=v["d_length"], d_parent=v["d_parent"], stream=0)


def refused(code, call, **kw):
    with pytest.raises(gdn.GdnError) as e:
        call(**kw)
    assert e.value.status == code and str(e.value), kw


@pytest.mark.parametrize("kw", BAD_DIMS)
def test_dims(kw):
    refused(gdn.GDN_ERR_SHAPE, call_append, d=dims(**kw))
    refused(gdn.GDN_ERR_SHAPE, call_attend, d=dims(**kw))
    assert gdn.gdn_attend_workspace_bytes(dims(**kw)) == 0


def test_dtype():
    for call in (call_append, call_attend):
        refused(gdn.GDN_ERR_DTYPE, call, d=dims(dtype=5))


@pytest.mark.parametrize("name", ["k", "v", "page_table", "past"])
def test_cache(name):
    for call in (call_append, call_attend):
        refused(gdn.GDN_ERR_ARG, call, c=cache(**{name: None}))
        refused(gdn.GDN_ERR_ALIGN, call, c=cache(**{name: A + 8}))


def test_null_structs():
    L = gdn.lib()
    d, c, p = dims(), cache(), gdn.qk_params(32, A)
    r = ctypes.byref
    assert L.gdn_kv_append(None, r(c), r(p), A, A, A, 512, 128, 128, A, None, None, None, None, None) == gdn.GDN_ERR_ARG
    assert L.gdn_kv_append(r(d), None, r(p), A, A, A, 512, 128, 128, A, None, None, None, None, None) == gdn.GDN_ERR_ARG
    assert L.gdn_kv_append(r(d), r(c), None, A, A, A, 512, 128, 128, A, None, None, None, None, None) == gdn.GDN_ERR_ARG
    assert L.gdn_attend(r(d), r(c), None, A, A, None, None, A, 1 << 40, None, None) == gdn.GDN_ERR_ARG
    assert L.gdn_attend(None, r(c), None, A, A, None, None, A, 1 << 40, None, None) == gdn.GDN_ERR_ARG
    assert L.gdn_attend_workspace_bytes(None) == 0


@pytest.mark.parametrize("code,kw", [
    (gdn.GDN_ERR_ARG, dict(k=None)), (gdn.GDN_ERR_ARG, dict(v=None)), (gdn.GDN_ERR_ARG, dict(q=None)),
    (gdn.GDN_ERR_ARG, dict(q_out=None)), (gdn.GDN_ERR_ARG, dict(d_path=A)), (gdn.GDN_ERR_ARG, dict(d_path=A, d_parent=A)),
    (gdn.GDN_ERR_ARG, dict(d_path=A, d_parent=A, q=None, q_out=None)),
    (gdn.GDN_ERR_SHAPE, dict(ld_q=504)), (gdn.GDN_ERR_SHAPE, dict(ld_k=120)), (gdn.GDN_ERR_SHAPE, dict(ld_v=132)),
    (gdn.GDN_ERR_SHAPE, dict(ld_q=-512)), (gdn.GDN_ERR_SHAPE, dict(ld_q=2 ** 38)),
    (gdn.GDN_ERR_SHAPE, dict(q_out=A, ld_q=520)),
    (gdn.GDN_ERR_SHAPE, dict(d=dims(n_tokens=65), d_parent=A)),
    (gdn.GDN_ERR_SHAPE, dict(p=gdn.qk_params(80, A))), (gdn.GDN_ERR_SHAPE, dict(p=gdn.qk_params(24, A))),
    (gdn.GDN_ERR_SHAPE, dict(p=gdn.qk_params(-16, A))), (gdn.GDN_ERR_ARG, dict(p=gdn.qk_params(32, None))),
    (gdn.GDN_ERR_ARG, dict(p=gdn.qk_params(32, A, norm_eps=-1.0))), (gdn.GDN_ERR_ARG, dict(p=gdn.qk_params(32, A, norm_eps=math.nan))),
    (gdn.GDN_ERR_ALIGN, dict(q=A + 2)), (gdn.GDN_ERR_ALIGN, dict(k=A + 2)), (gdn.GDN_ERR_ALIGN, dict(v=A + 4)),
    (gdn.GDN_ERR_ALIGN, dict(q_out=A + 8)), (gdn.GDN_ERR_ALIGN, dict(d_length=A + 4)), (gdn.GDN_ERR_ALIGN, dict(d_parent=A + 4)),
    (gdn.GDN_ERR_ALIGN, dict(p=gdn.qk_params(32, A + 4))), (gdn.GDN_ERR_ALIGN, dict(p=gdn.qk_params(32, A, A + 4))),
    (gdn.GDN_ERR_ALIGN, dict(q=None, q_out=None, d_path=A + 4)),
])
def test_append(code, kw):
    refused(code, call_append, **kw)


@pytest.mark.parametrize("code,kw", [
    (gdn.GDN_ERR_ARG, dict(q=None)), (gdn.GDN_ERR_ARG, dict(out=None)), (gdn.GDN_ERR_ARG, dict(out=A)),
    (gdn.GDN_ERR_ARG, dict(p=gdn.attn_params(math.nan))), (gdn.GDN_ERR_ARG, dict(p=gdn.attn_params(math.inf))),
    (gdn.GDN_ERR_ARG, dict(p=gdn.attn_params(1.0, -1))), (gdn.GDN_ERR_ARG, dict(p=gdn.attn_params(1.0, 5, -1))),
    (gdn.GDN_ERR_SHAPE, dict(d=dims(n_tokens=65), d_parent=A)),
    (gdn.GDN_ERR_ALIGN, dict(q=A + 2)), (gdn.GDN_ERR_ALIGN, dict(out=A + 8)), (gdn.GDN_ERR_ALIGN, dict(d_length=A + 4)),
    (gdn.GDN_ERR_ALIGN, dict(d_parent=A + 4)), (gdn.GDN_ERR_ALIGN, dict(workspace=A + 16)),
    (gdn.GDN_ERR_WORKSPACE, dict(workspace=None)), (gdn.GDN_ERR_WORKSPACE, dict(ws_bytes=0)),
])
def test_attend(code, kw):
    refused(code, call_attend, **kw)


@pytest.mark.parametrize("dtype", [gdn.GDN_F32, gdn.GDN_BF16])
def test_more_work_than_a_launch_counts(dtype):
    """Blocks of rows times kv heads times key tiles past 2^31."""
    kw = dict(n_slots=2 ** 10, n_tokens=2 ** 10, n_heads=64, n_kv_heads=64, page_tokens=256, max_pages=2 ** 12, dtype=dtype)
    refused(gdn.GDN_ERR_SHAPE, call_attend, d=dims(**kw))
    assert gdn.gdn_attend_workspace_bytes(dims(**kw)) == 0
    assert gdn.gdn_attend_workspace_bytes(dims(**{**kw, "n_slots": 1})) > 0


def test_workspace_is_asked_for_in_full():
    for dtype in (gdn.GDN_F32, gdn.GDN_BF16):
        d = dims(dtype=dtype)
        need = gdn.gdn_attend_workspace_bytes(d)
        assert 0 < need < 1 << 28
        refused(gdn.GDN_ERR_WORKSPACE, call_attend, d=d, ws_bytes=need - 1)
