"""GPU parity of hs_batch_plan against the oracle: whole numbers, all equal."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import chunk as C  # noqa: E402

pytestmark = pytest.mark.gpu
NAMES = ("token_offsets", "seq_lens", "entries", "positions", "rows", "block_tables")


def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hierarchical_sparse_attention_gb300 as hs
    return hs


def d(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def call(hs, req, old, new, table, page, pool_rows, max_tokens, max_blocks, leave=(), stream=None):
    n = len(req)
    size = {"token_offsets": n + 1, "seq_lens": n, "block_tables": n * (max_blocks or 0)}
    out = {k: torch.full((size.get(k, max_tokens),), -77, dtype=torch.int32, device="cuda") for k in NAMES if k not in leave}
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = [d(np.asarray(x, np.int32)) for x in (req, old, new)]
    hs.hs_batch_plan(n, *i32, table.shape[0], d(table), table.shape[1], page, pool_rows, max_tokens, *[out.get(k) for k in NAMES[:5]], max_blocks or 1, out.get("block_tables"), err,
                     stream)
    return {k: v.cpu().numpy() for k, v in out.items()}, int(err.item())


def check(hs, req, old, new, table, page, pool_rows, max_tokens, max_blocks):
    leave = () if max_blocks else ("block_tables",)
    got, flags = call(hs, req, old, new, table, page, pool_rows, max_tokens, max_blocks, leave)
    want, wflags = C.plan(req, old, new, table, page, pool_rows, max_tokens, max_blocks)
    for k in want:
        assert np.array_equal(got[k], want[k].reshape(-1)), k
    assert flags == wflags


@pytest.mark.parametrize("n,slots,page,most,room", [(1, 1, 1, 3, 0), (1, 4, 64, 200, 5), (7, 9, 16, 90, 0), (32, 40, 64, 1, 3), (511, 600, 64, 5, 0), (512, 512, 48, 4, 9), (513, 700, 16, 6, 2),
                                                    (1300, 2000, 7, 9, 700)])
def test_batches_of_many_kinds(n, slots, page, most, room):
    hs = _gpu()
    rng = np.random.default_rng(n * 7 + page)
    max_pages = 300 // page + 40
    table = np.full((slots, max_pages), -1, np.int32)
    table[:] = rng.permutation(slots * max_pages).reshape(slots, max_pages)
    table[rng.random(table.shape) < 0.01] = -1
    req = rng.permutation(slots)[:n].astype(np.int32)
    old = rng.integers(0, 300, n)
    new = old + rng.integers(0, most + 1, n)
    req[rng.random(n) < 0.05] = -3
    total = int((new - old)[req >= 0].sum())
    check(hs, req, old, new, table, page, slots * max_pages * page, total + room, -(-int(new.max()) // page) + 2)
    check(hs, req, old, new, table, page, slots * max_pages * page // 2, total + room, None)


def test_refused_entries():
    hs = _gpu()
    rng = np.random.default_rng(3)
    table = rng.permutation(8 * 10).reshape(8, 10).astype(np.int32)
    req = [3, 9, 5, 3, 0, 1, 2, -1, 4, 7]
    old = [0, 0, 4, 0, 7, -1, 0, 0, 3, 2]
    new = [5, 2, 4, 5, 6, 3, 161, 9, 9, 4]
    for room in (8, 7, 6, 5, 1, 0):  # the last two entries of 6 and 2 tokens: both, one, none
        check(hs, req, old, new, table, 16, 10000, room, 10)
    check(hs, req, old, new, table, 16, 10000, 40, 1)  # block tables of one page
    check(hs, [2 ** 31 - 1, -2 ** 31], [0, 0], [2 ** 31 - 1, 1], table, 16, 10000, 4, 10)
    check(hs, [1, 2, 3], [2 ** 31 - 1, 0, 1], [2 ** 31 - 1, 160, 160], table, 16, 2 ** 31 - 1, 400, 12)


def test_nothing_in_the_batch_and_outputs_left_out():
    hs = _gpu()
    table = np.zeros((2, 3), np.int32)
    got, flags = call(hs, [], [], [], table, 4, 100, 5, 2)
    assert got["token_offsets"].tolist() == [0] and all((got[k] == -1).all() for k in ("entries", "positions", "rows")) and flags == 0
    full, _ = call(hs, [1, 0], [0, 2], [3, 4], table, 4, 100, 9, 2)
    for leave in NAMES[1:]:
        got, _ = call(hs, [1, 0], [0, 2], [3, 4], table, 4, 100, 9, 2, (leave,))
        assert all(np.array_equal(got[k], full[k]) for k in got)


def test_a_page_of_the_last_rows():
    hs = _gpu()
    page = 64
    last = (2 ** 31 - 1) // page  # its rows begin at 2^31 - 64
    table = np.array([[last, last + 1, 2 ** 31 - 1]], np.int32)
    check(hs, [0], [60], [190], table, page, 2 ** 31 - 1, 140, 3)


def test_captured_and_replayed_with_other_lengths():
    hs = _gpu()
    rng = np.random.default_rng(4)
    n, page, room = 40, 16, 200
    table = rng.permutation(50 * 12).reshape(50, 12).astype(np.int32)
    ins = [torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(3)]
    outs = [torch.zeros(k, dtype=torch.int32, device="cuda") for k in (n + 1, n, room, room, room, n * 12)]
    err, tab = torch.zeros(1, dtype=torch.int32, device="cuda"), d(table)
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        hs.hs_batch_plan(n, *ins, 50, tab, 12, page, 9600, room, *outs[:5], 12, outs[5], err, side)
    for _ in range(3):
        req, old = rng.permutation(50)[:n], rng.integers(0, 150, n)
        new = old + rng.integers(0, 9, n)
        for t, x in zip(ins, (req, old, new)):
            t.copy_(d(x.astype(np.int32)))
        g.replay()
        want, _ = C.plan(req, old, new, table, page, 9600, room, 12)
        for k, o in zip(NAMES, outs):
            assert np.array_equal(o.cpu().numpy(), want[k].reshape(-1)), k
