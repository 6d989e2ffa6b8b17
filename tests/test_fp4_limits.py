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
