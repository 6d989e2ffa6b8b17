"""The 4-bit calls where a CTA pair goes through several units, calls follow one another closely, run at
once or from graphs, and at the ends of their ranges. Tolerances: test_gpu_fp4's, derived there."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import test_gpu_fp4 as T  # noqa: E402
import test_gpu_pages as G  # noqa: E402
from oracle import fp4_mla as F  # noqa: E402

pytestmark = pytest.mark.gpu


def ragged(rng, n):
    """Lengths whose numbers of blocks follow each other as 0, 1, 2, 3, many, in every order."""
    return rng.choice([0, 1, 5, 63, 64, 65, 128, 129, 192, 200, 330, 900], n).astype(np.int32)


@pytest.mark.parametrize("H,Q,W,sinks,splits,R", [(128, 1, 5000, 0, 1, 260), (128, 1, 300, 5, 1, 400), (16, 4, 700, 3, 1, 300),
                                                  (128, 2, 200, 4, 3, 90), (100, 1, 64, 0, 5, 150), (128, 1, 1, 0, 1, 500),
                                                  (128, 3, 200, 4, 3, 60), (40, 4, 300, 0, 2, 120)])
def test_pairs_go_through_units_of_every_length(H, Q, W, sinks, splits, R):
    hs = T._gpu()
    rng = np.random.default_rng(R + W)
    lens = ragged(rng, R)
    table, rows = T.pages_for(rng, lens, 16, 60)
    q, pool, _ = T.case(R, R, H, 1, rows, g=0.5, Q=Q)
    q[lens == 0] = 0x7FC0  # what a padded request's q holds does not matter
    o, lse, err = T.window(hs, q, T.d(pool), 16, lens, table, W, sinks, 0.5, splits)
    assert err == 0
    T.check_window(q, pool, 16, lens, table, W, sinks, 0.5, o, lse)


@pytest.mark.parametrize("K,splits", [(64, 1), (1, 1), (130, 1), (320, 2)])
def test_many_sparse_units_with_empty_ones_between(K, splits):
    hs = T._gpu()
    q, pool, rows = T.case(K, 330, 128, K, 900, masked=0.3)
    rows[::3] = -1
    q[::3] = 0x7FC0  # NaN, where there is no row to look at
    o, lse, err = T.sparse(hs, q, T.d(pool), T.d(rows), 1.0, splits)
    assert err == 0
    for r in range(330):
        T.check(q[r], pool[rows[r][rows[r] >= 0]], 1.0, o[r], lse[r], f"request {r}")


@pytest.mark.parametrize("sm", [-0.05, 0.0, 1e-30])
@pytest.mark.parametrize("splits", [1, 3])
def test_scales_of_either_sign_and_zero(sm, splits):
    hs = T._gpu()
    q, pool, rows = T.case(11, 3, 30, 300, 400, g=4.0)
    rows[2] = -1
    o, lse, err = T.sparse(hs, q, T.d(pool), T.d(rows), 4.0, splits, sm)
    assert err == 0
    for r in range(3):
        T.check(q[r], pool[rows[r][rows[r] >= 0]], 4.0, o[r], lse[r], f"request {r}", sm)


def test_references_that_are_passed_by_little_and_by_much():
    """Scores that creep up by a few powers of two a block (the reference stays), jump by dozens (it
    moves) and come from rows of which each head sees others first: the weights stay in f16's range."""
    hs = T._gpu()
    rng = np.random.default_rng(21)
    n = 64 * 40
    kv = np.zeros((n, 576))
    kv[:, :512] = rng.standard_normal((n, 512))
    blk = np.arange(n) // 64
    kv[:, 512] = blk * 0.5
    kv[:, 513] = np.where(blk == 17, 4, 0) + np.where(blk == 30, 16, 0)
    kv[:, 514] = (39 - blk) * 0.5
    pool = F.pack(T.bf16_bits(kv), 1.0)
    q = rng.standard_normal((2, 128, 576)) * 0.3
    q[:, :, 512:515] = rng.choice([0.0, 1.0, 4.0, 16.0], (2, 128, 3))
    q = T.bf16_bits(q)
    rows = np.stack([np.arange(n), np.arange(n)[::-1]]).astype(np.int32).copy()
    for splits in (1, 2, 16):
        o, lse, err = T.sparse(hs, q, T.d(pool), T.d(rows), 1.0, splits, 1.0)
        assert err == 0
        for r in range(2):
            T.check(q[r], pool[rows[r]], 1.0, o[r], lse[r], f"request {r}, {splits} splits", 1.0)


def test_outputs_and_workspaces_on_16_byte_boundaries():
    hs = T._gpu()
    q, pool, rows = T.case(31, 3, 100, 300, 400)
    dq, dp, dr = T.d(q), T.d(pool), T.d(rows)
    for splits in (1, 3):
        want = T.sparse(hs, q, dp, dr, 1.0, splits)
        wsb = hs.hs_fp4_mla_workspace_bytes(3, 100, 1, splits)
        ws = torch.empty(wsb + 32, dtype=torch.uint8, device="cuda")[16:]
        raw = torch.full((3 * 100 * 512 + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
        o, lse, err = raw[8:-8].view(3, 100, 512), torch.zeros(3, 100, device="cuda"), T.flags()
        assert o.data_ptr() % 32 == 16 and ws.data_ptr() % 32 == 16
        hs.hs_fp4_sparse_mla_decode(3, 100, 300, splits, dq, dp, 400, dr, T.SM, 1.0, o, lse, ws, wsb, err)
        assert np.array_equal(o.float().cpu().numpy(), want[0]) and np.array_equal(lse.cpu().numpy(), want[1])
        assert (raw[:8] == 7).all() and (raw[-8:] == 7).all() and int(err.item()) == 0


def test_calls_close_together_repeat_their_results():
    """Calls of different shapes one after the other, over a shared workspace: each may begin while the
    one before it ends. Every repetition gives the same bits."""
    hs = T._gpu()
    rng = np.random.default_rng(41)
    lens = ragged(rng, 100)
    table, rows = T.pages_for(rng, lens, 16, 60)
    pool = T.d(T.case(1, 1, 1, 1, rows)[1])
    dl, dt, err = T.d(lens), T.d(table), T.flags()
    kinds = []
    for R, H, K, splits in ((100, 128, 200, 1), (3, 128, 1000, 8), (100, 16, 64, 2)):
        q, _, tab = T.case(R + H, R, H, K, 100)
        kinds.append((R, H, K, splits, T.d(q), T.d(tab)))
    q = T.d(T.case(9, 100, 32, 1, 10, Q=3)[0])
    wsb = max([hs.hs_fp4_mla_workspace_bytes(k[0], k[1], 1, k[3]) for k in kinds] + [hs.hs_fp4_mla_workspace_bytes(100, 32, 3, 2)])
    ws = torch.zeros(wsb, dtype=torch.uint8, device="cuda")
    buffers = [(torch.empty(100, 128, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(100, 128, device="cuda")) for _ in range(4)]

    def calls():
        for (o, lse), (R, H, K, splits, dq, dtab) in zip(buffers, kinds):
            hs.hs_fp4_sparse_mla_decode(R, H, K, splits, dq, pool, rows, dtab, T.SM, 1.0, o, lse, ws, wsb, err)
        hs.hs_fp4_window_mla_decode(100, 32, 3, 250, 2, 2, q, pool, rows, 16, 60, dl, dt, T.SM, 1.0, *buffers[3], ws, wsb, err)

    calls()
    first = [x.clone() for b in buffers for x in b]
    for _ in range(40):
        calls()
        calls()
        for x, y in zip(first, (x for b in buffers for x in b)):
            assert torch.equal(x.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32),
                               y.view(torch.int16 if y.dtype == torch.bfloat16 else torch.int32))
    assert int(err.item()) == 0


def test_two_streams_at_once():
    hs = T._gpu()
    q, pool, rows = T.case(51, 120, 128, 256, 2000)
    dq, dp, dr = T.d(q), T.d(pool), T.d(rows)
    wsb = hs.hs_fp4_mla_workspace_bytes(120, 128, 1, 3)
    out = []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for s, splits in zip(streams, (1, 3)):
        o = torch.empty(120, 128, 512, dtype=torch.bfloat16, device="cuda")
        out.append((o, torch.empty(120, 128, device="cuda"), torch.empty(wsb, dtype=torch.uint8, device="cuda"), T.flags()))
    torch.cuda.synchronize()
    for _ in range(10):
        for s, splits, (o, lse, ws, err) in zip(streams, (1, 3), out):
            hs.hs_fp4_sparse_mla_decode(120, 128, 256, splits, dq, dp, 2000, dr, T.SM, 1.0, o, lse, ws, wsb, err, stream=s)
    torch.cuda.synchronize()
    for splits, (o, lse, _, err) in zip((1, 3), out):
        assert int(err.item()) == 0
        want = T.sparse(hs, q, dp, dr, 1.0, splits)
        assert np.array_equal(o.float().cpu().numpy(), want[0]) and np.array_equal(lse.cpu().numpy(), want[1])


def test_a_step_captured_behind_copies_and_another_stream():
    """pack, attention, unpack and page calls in one graph, their inputs from a copy node and from a kernel
    of a second captured stream: replayed with new tokens, they see them."""
    hs = T._gpu()
    rng = np.random.default_rng(61)
    R, ps = 4, 16
    s = G.Pair(hs, 8, 8, 6, 40, ps)
    s.extend([0, 1, 2, 3], [0] * 4, [40, 17, 16, 60])
    lens = np.array([40, 17, 16, 60], np.int32)
    pool, total = s.pools[0], 40 * ps
    all_rows = np.concatenate([s.orc.table[r, np.arange(n) // ps] * ps + np.arange(n) % ps for r, n in enumerate(lens)]).astype(np.int32)
    n = all_rows.size
    staged = torch.zeros(n, 576, dtype=torch.int16, device="cuda")  # the graph's inputs
    kv, rows, q0 = torch.zeros_like(staged), torch.zeros(n, dtype=torch.int32, device="cuda"), d_q(rng, R)
    row_src, dl = T.d(all_rows), T.d(lens)
    o, lse = torch.zeros(R, 1, 16, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(R, 1, 16, device="cuda")
    back = torch.zeros(n, 576, dtype=torch.int16, device="cuda")
    fork = [T.d(np.array(x, np.int32)) for x in ([0, 3], [4, 5], [40, 60])]
    side, main, g = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=main):
        kv.copy_(staged)  # a copy node
        side.wait_stream(main)
        with torch.cuda.stream(side):
            rows.copy_(row_src + 0)
        main.wait_stream(side)  # two nodes before the first call
        hs.hs_fp4_pack_rows(n, kv, 576, rows, 1.0, pool, total, s.err, stream=main)
        hs.hs_fp4_window_mla_decode(R, 16, 1, 1000, 0, 1, q0, pool, total, ps, 6, dl, s.table, T.SM, 1.0, o, lse, None, 0, s.err, stream=main)
        hs.hs_pages_fork(s.pool, 2, *fork, None, main)
        hs.hs_fp4_unpack_rows(n, pool, total, rows, 1.0, back, 576, s.err, stream=main)
        hs.hs_pages_free(s.pool, 1, fork[1][:1], None, None, main)
        hs.hs_pages_free(s.pool, 1, fork[1][1:], None, None, main)
    for _ in range(3):
        new = T.tokens(rng, n)
        staged.copy_(T.d(new))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        rec = F.pack(new, 1.0)
        qq = q0.cpu().numpy().view(np.uint16)
        at = 0
        for r, k in enumerate(lens):
            T.check(qq[r, 0], rec[at:at + k], 1.0, o[r, 0].float().cpu().numpy(), lse[r, 0].cpu().numpy(), f"request {r}")
            at += k
        want = np.concatenate(F.unpack(rec, 1.0), 1)
        assert np.array_equal(F.bf16_decode(back.cpu().numpy().view(np.uint16)), want)
        assert np.array_equal(s.table.cpu().numpy(), s.orc.table) and int(s.count.item()) == len(s.orc.free) and int(s.err.item()) == 0


def d_q(rng, R):
    return T.d(T.bf16_bits(rng.standard_normal((R, 1, 16, 576))))


def test_a_window_at_the_end_of_a_sequence_of_two_billion_tokens():
    """Token numbers up to 2^31 - 2 and pages of 2^20 rows; the last row of the pool is a token's."""
    hs = T._gpu()
    rng = np.random.default_rng(71)
    page, pages = 1 << 20, 2047
    total = page * 2
    pool = torch.zeros(total, 416, dtype=torch.uint8, device="cuda")
    rec = F.pack(T.tokens(rng, 300), 1.0)
    pool[total - 300:] = torch.from_numpy(rec).cuda()  # the end of page 1
    table = np.full((2, pages), -1, np.int32)
    table[0, pages - 1] = 1
    table[1, 0] = 1
    lens = np.array([pages * page, page], np.int32)
    q = T.bf16_bits(rng.standard_normal((2, 2, 20, 576)))
    o, lse, err = T.window(hs, q, pool, page, lens, table, 150, 0, 1.0, 2)
    assert err == 0
    for r in range(2):
        for i in range(2):
            T.check(q[r, i], rec[300 - 151 + i:300 - 1 + i], 1.0, o[r, i], lse[r, i], f"request {r} query {i}")
    table[0, pages - 1] = 2  # a page past the pool
    o, lse, err = T.window(hs, q, pool, page, lens, table, 150, 0, 1.0, 1)
    assert err == hs.HS_FLAG_DEVROW and (o[0] == 0).all() and np.isneginf(lse[0]).all()


@pytest.mark.parametrize("page,row_bytes,layers,skew", [(64, 416, 2, 0), (100, 656, 1, 0), (64, 416, 1, 4)])
def test_compaction_of_many_large_pages(page, row_bytes, layers, skew):
    """Pages of several spans, more of them than the copying warps' rings hold."""
    hs = T._gpu()
    rng = np.random.default_rng(page + layers)
    s = G.Pair(hs, 9, 400, 8, 3000, page, row_bytes, layers, skew)
    s.extend(list(range(370)), [0] * 370, [8 * page] * 370)
    s.release(rng.permutation(370)[:150].tolist())
    s.compact()
    s.extend([399], [0], [8 * page])
    s.release(rng.permutation(370)[:150].tolist())
    s.compact()


def test_the_most_requests():
    hs = T._gpu()
    n = hs.HS_MAX_PAGE_REQUESTS
    rng = np.random.default_rng(3)
    s = G.Pair(hs, 10, n, 2, n + 3000, 1, 1)
    r = rng.permutation(n)[:n // 2 + 5000]
    s.extend(r.tolist(), [0] * r.size, rng.integers(0, 3, r.size).tolist())
    idle = np.flatnonzero((s.orc.table == -1).all(1))
    busy = np.flatnonzero((s.orc.table != -1).all(1))
    k = min(idle.size, 20000)
    s.fork(rng.choice(busy, k).tolist(), idle[:k].tolist(), rng.integers(0, 3, k).tolist())
    s.release(list(range(n)) + list(range(0, n, 7)))
    s.compact()
    assert int(s.count.item()) == n + 3000


def test_strides_that_do_not_fit_are_refused():
    hs = T._gpu()
    kv, pool = torch.zeros(8, 640, dtype=torch.int16, device="cuda"), torch.zeros(100, 416, dtype=torch.uint8, device="cuda")
    rows, err = torch.arange(8, dtype=torch.int32, device="cuda"), T.flags()
    hs.hs_fp4_pack_rows(8, kv[:, :576], 640, rows, 1.0, pool, 100, err)
    hs.hs_fp4_pack_rows(1, kv[:1, :576], 576, rows, 1.0, pool, 100, err)  # one row: its stride says nothing
    q = torch.zeros(2, 16, 1152, dtype=torch.bfloat16, device="cuda")
    o, lse = torch.zeros(2, 16, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 16, device="cuda")
    for call in (lambda: hs.hs_fp4_pack_rows(8, kv[:, :576], 576, rows, 1.0, pool, 100, err),
                 lambda: hs.hs_fp4_pack_rows(8, kv.t(), 640, rows, 1.0, pool, 100, err),
                 lambda: hs.hs_fp4_pack_rows(4, kv[:, :576], 640, rows[::2], 1.0, pool, 100, err),
                 lambda: hs.hs_fp4_unpack_rows(8, pool[:, :400], 100, rows, 1.0, kv, 640, err),
                 lambda: hs.hs_fp4_sparse_mla_decode(2, 16, 4, 1, q[:, :, :576], pool, 100, rows.view(2, 4), 0.1, 1.0, o, lse, None, 0, err)):
        with pytest.raises(ValueError):
            call()
    assert int(err.item()) == 0
