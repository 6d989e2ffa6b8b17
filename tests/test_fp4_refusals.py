"""Calls on 4-bit rows and pages that the host refuses: sizes and scales past the documented ends."""
import pytest

A = 1 << 20  # an aligned stand-in address: nothing is launched in these calls


def test_page_calls_of_too_many_entries_are_refused():
    import hierarchical_sparse_attention_gb300 as hs
    p = hs.make_page_pool([A], 4, 8, 100, 16, 416, A, A, A, A, A, hs.hs_pages_workspace_bytes(4, 100), A)
    n = hs.HS_MAX_PAGE_ENTRIES + 1
    for call in (lambda: hs.hs_pages_extend(p, n, A, A, A), lambda: hs.hs_pages_free(p, n, A),
                 lambda: hs.hs_pages_extend(p, 2 ** 31 - 1, A, A, A), lambda: hs.hs_pages_free(p, 2 ** 31 - 1, A)):
        with pytest.raises(hs.HsError) as e:
            call()
        assert e.value.status == hs.HS_ERR_INVALID_ARG


@pytest.mark.parametrize("sm,g", [(3e38, 2.0), (1e30, 2.0 ** 32), (-3e38, 1.5 * 2), (2.5e38, 1.0)])
def test_scales_whose_product_is_infinite_are_refused(sm, g):
    import hierarchical_sparse_attention_gb300 as hs
    for call in (lambda: hs.hs_fp4_sparse_mla_decode(2, 16, 64, 1, A, A, 100, A, sm, g, A, A, None, 0, A),
                 lambda: hs.hs_fp4_window_mla_decode(2, 16, 1, 8, 1, 1, A, A, 100, 16, 8, A, A, sm, g, A, A, None, 0, A)):
        with pytest.raises(hs.HsError) as e:
            call()
        assert e.value.status == hs.HS_ERR_INVALID_ARG


def test_arrays_off_the_device_are_refused_by_every_call():
    """Host tensors and arrays, and rows that are not as far apart as the call says."""
    np = pytest.importorskip("numpy")
    torch = pytest.importorskip("torch")
    import hierarchical_sparse_attention_gb300 as hs
    for x in (torch.zeros(8, 576, dtype=torch.int16), np.zeros((8, 576), np.int16)):
        for call in (lambda: hs.hs_fp4_pack_rows(8, x, 576, A, 1.0, A, 100, A),
                     lambda: hs.hs_fp4_pack_rows(8, A, 576, x, 1.0, A, 100, A),
                     lambda: hs.hs_fp4_unpack_rows(8, A, 100, A, 1.0, x, 576, A),
                     lambda: hs.hs_fp4_sparse_mla_decode(2, 16, 64, 1, x, A, 100, A, 0.1, 1.0, A, A, None, 0, A),
                     lambda: hs.hs_fp4_window_mla_decode(2, 16, 1, 8, 1, 1, A, A, 100, 16, 8, A, x, 0.1, 1.0, A, A, None, 0, A),
                     lambda: hs.make_page_pool([A], 4, 8, 100, 16, 416, A, x, A, A, A, 1 << 20, A)):
            with pytest.raises(ValueError):
                call()
