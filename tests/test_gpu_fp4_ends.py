"""The 4-bit calls at the far ends of what their documentation allows: the most pages, scores of any size, weights
of any size. Tolerances: test_gpu_fp4's terms, or derived here."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import test_gpu_fp4 as T  # noqa: E402
from oracle import fp4_mla as F  # noqa: E402

pytestmark = pytest.mark.gpu


def test_the_most_pages_a_pool_can_have():
    """2^31 - 1 pages of one row of a byte: the number of 32-page words passes what 32 bits hold before the
    division. The workspace holds ones before the call that makes it ready."""
    hs = T._gpu()
    n = 2 ** 31 - 1
    wsb = hs.hs_pages_workspace_bytes(1, n)
    if torch.cuda.mem_get_info()[0] < 2 * 4 * n + wsb + n + (4 << 30):
        pytest.skip("needs 46 GB of device memory")
    table = torch.full((1, 4), 7, dtype=torch.int32, device="cuda")
    refs, free = (torch.empty(n, dtype=torch.int32, device="cuda") for _ in range(2))
    refs[-64:], free[-64:] = 77, 77
    count, err = T.flags(), T.flags()
    ws, pool = torch.empty(wsb, dtype=torch.uint8, device="cuda"), torch.empty(n, 1, dtype=torch.uint8, device="cuda")
    words = (n + 31) // 32
    ws[:256 + 4 * words] = 255
    p = hs.make_page_pool([pool], 1, 4, n, 1, 1, table, refs, free, count, ws, wsb, err)
    hs.hs_pages_init(p)
    marks = ws[256:256 + 4 * words].view(torch.int32)
    assert not marks.any()
    assert int(count.item()) == n and free[[0, n - 1]].tolist() == [n - 1, 0] and int(refs[-1]) == 0 and (table == -1).all()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    hs.hs_pages_extend(p, 1, i32(0), i32(0), i32(3), None)
    assert table.tolist() == [[0, 1, 2, -1]] and int(count.item()) == n - 3
    hs.hs_pages_free(p, 1, i32(0), i32(1), None)
    assert table.tolist() == [[0, -1, -1, -1]] and int(count.item()) == n - 1 and free[n - 3:n - 1].tolist() == [2, 1]
    assert not marks.any() and int(err.item()) == 0
