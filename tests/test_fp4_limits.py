"""The 4-bit calls' limits as include/hs.h names them, and refusals that no other check comes before (no GPU)."""
import os
import re

import pytest

A = 1 << 20  # an aligned stand-in address: nothing is launched in these calls
HEADER = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "hs.h")).read()


def defined(name):
    return eval(re.search(r"#define %s\s+(\(.*?\)|\d+)" % name, HEADER).group(1), {})


def test_the_most_requests_of_an_attention_call_are_documented():
    import hierarchical_sparse_attention_gb300 as hs
    most = defined("HS_MAX_FP4_MLA_REQUESTS")
    assert most == hs.HS_MAX_FP4_MLA_REQUESTS
    assert hs.hs_fp4_mla_workspace_bytes(most, 1, 1, 2) > 0 and hs.hs_fp4_mla_workspace_bytes(most + 1, 1, 1, 2) == 0
    for call in (lambda r: hs.hs_fp4_sparse_mla_decode(r, 16, 64, 1, A, A, 100, A, 0.1, 1.0, A, A, None, 0, A),
                 lambda r: hs.hs_fp4_window_mla_decode(r, 16, 1, 8, 1, 1, A, A, 100, 16, 8, A, A, 0.1, 1.0, A, A, None, 0, A)):
        with pytest.raises(hs.HsError) as e:
            call(most + 1)
        assert e.value.status == hs.HS_ERR_INVALID_ARG


@pytest.mark.parametrize("sm,g", [(-3e38, 2.0), (-1e30, 2.0 ** 32), (-2.5e38, 1.0)])
def test_scales_whose_product_is_negative_and_infinite_are_refused(sm, g):
    """Scales that are allowed each for itself, so that only their product can be the reason."""
    import hierarchical_sparse_attention_gb300 as hs
    for call in (lambda: hs.hs_fp4_sparse_mla_decode(2, 16, 64, 1, A, A, 100, A, sm, g, A, A, None, 0, A),
                 lambda: hs.hs_fp4_window_mla_decode(2, 16, 1, 8, 1, 1, A, A, 100, 16, 8, A, A, sm, g, A, A, None, 0, A)):
        with pytest.raises(hs.HsError) as e:
            call()
        assert e.value.status == hs.HS_ERR_INVALID_ARG
    hs.hs_fp4_sparse_mla_decode(0, 16, 64, 1, None, None, 100, None, 0.1, g, None, None, None, 0, None)
    hs.hs_fp4_sparse_mla_decode(0, 16, 64, 1, None, None, 100, None, -1e4, 1.0, None, None, None, 0, None)


def test_page_calls_refuse_entries_off_the_device():
    np = pytest.importorskip("numpy")
    torch = pytest.importorskip("torch")
    import hierarchical_sparse_attention_gb300 as hs
    p = hs.make_page_pool([A], 4, 8, 100, 16, 416, A, A, A, A, A, hs.hs_pages_workspace_bytes(4, 100), A)
    for x in (torch.zeros(4, dtype=torch.int32), np.zeros(4, np.int32)):
        for call, n in ((hs.hs_pages_extend, 4), (hs.hs_pages_fork, 4), (hs.hs_pages_free, 3)):
            for i in range(n):
                with pytest.raises(ValueError):
                    call(p, 1, *[x if k == i else A for k in range(n)])
