"""Limits of gdn_attend as its header states them (no GPU needed): the largest work that a launch counts, asked of the
workspace, and the largest scale."""
import pytest

import gated_deltanet_verify_gb300 as gdn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build_library()


def counted(B, T, G, Hk, D, page, max_pages, dtype):
    """Blocks of rows times kv heads times key tiles."""
    sizes, last = ([32], 128) if dtype == gdn.GDN_BF16 else ([8, 16, 32], 64)
    r = next((r for r in sizes if T * G <= r), last)
    b = min(T, r // G)
    tiles = -(-max_pages * page // (128 if dtype == gdn.GDN_BF16 else 32)) + ((4 if D == 64 else 3) if dtype == gdn.GDN_BF16 else 0)
    return B * -(-T // b) * Hk * tiles


@pytest.mark.parametrize("dtype", [gdn.GDN_F32, gdn.GDN_BF16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,G", [(1, 1), (1, 8), (4, 8), (5, 7), (16, 6), (33, 1), (100, 48), (4096, 6)])
def test_the_limit_is_the_stated_one(T, G, D, dtype):
    Hk, page = 4, 256
    for B in (1, 64, 4096):
        if B * T > 2 ** 24:
            continue
        one = counted(B, T, G, Hk, D, page, 1, dtype)
        if one >= 2 ** 31:
            continue
        low, high = 1, 2 ** 30 // page             # the most pages that are below the limit
        while low < high:
            mid = (low + high + 1) // 2
            low, high = (mid, high) if counted(B, T, G, Hk, D, page, mid, dtype) < 2 ** 31 else (low, mid - 1)
        for max_pages in {1, low, min(low + 1, 2 ** 30 // page)}:
            dims = gdn.make_attn_dims(B, T, G * Hk, Hk, D, page, 10, max_pages, dtype=dtype)
            fits = counted(B, T, G, Hk, D, page, max_pages, dtype) < 2 ** 31
            assert (gdn.gdn_attend_workspace_bytes(dims) > 0) == fits, (B, max_pages)


def test_padding_counts():
    """One page of 128 positions is 1 + 4 tiles for heads of 64 in bf16."""
    kw = dict(n_tokens=1, n_heads=64, n_kv_heads=64, d_head=64, page_tokens=128, n_pages=1, max_pages=1, dtype=gdn.GDN_BF16)
    assert gdn.gdn_attend_workspace_bytes(gdn.make_attn_dims(n_slots=2 ** 24, **kw)) == 0
    assert gdn.gdn_attend_workspace_bytes(gdn.make_attn_dims(n_slots=2 ** 22, **kw)) > 0


@pytest.mark.parametrize("scale", [2.0 ** 126, -(2.0 ** 126), 3.4e38])
def test_scales_whose_powers_of_two_overflow_are_refused(scale):
    """Scores are taken to powers of two: scale times log2 e has to be a number, or a score of 0 would become NaN."""
    A = 0x10000
    dims = gdn.make_attn_dims(2, 4, 8, 2, 64, 16, 10, 5)
    with pytest.raises(gdn.GdnError) as e:
        gdn.gdn_attend(dims, gdn.kv_cache(A, A, A, A), gdn.attn_params(scale), A, A + 4096, A, 1 << 40, stream=0)
    assert e.value.status == gdn.GDN_ERR_ARG
