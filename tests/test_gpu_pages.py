"""GPU parity of the page calls against the oracle, bit for bit, and a run of them with the 4-bit rows
and the attention that reads them."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import fp4_mla as F  # noqa: E402
from oracle import pages as P  # noqa: E402

pytestmark = pytest.mark.gpu


def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hierarchical_sparse_attention_gb300 as hs
    return hs


def d(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


class Pair:
    """The same pool on the GPU and in the oracle, with canary bytes around the GPU's pools."""

    def __init__(self, hs, seed, requests, max_pages, pages, page_size, row_bytes=416, layers=1, skew=0):
        rng = np.random.default_rng(seed)
        rows = [rng.integers(0, 256, (pages * page_size, row_bytes)).astype(np.uint8) for _ in range(layers)]
        self.hs, self.skew, self.pages = hs, skew, pages
        self.orc = P.Pages(requests, max_pages, pages, page_size, rows)
        self.raw, self.pools = [], []
        for r in rows:
            raw = torch.full((r.size + 512,), 0xA7, dtype=torch.uint8, device="cuda")
            raw[256 + skew:256 + skew + r.size] = torch.from_numpy(r.reshape(-1)).cuda()
            self.raw.append(raw)
            self.pools.append(raw[256 + skew:256 + skew + r.size].view(r.shape))
        self.table = torch.full((requests, max_pages), 99, dtype=torch.int32, device="cuda")
        self.refs, self.free = (torch.full((pages,), 77, dtype=torch.int32, device="cuda") for _ in range(2))
        self.count, self.err = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
        wsb = hs.hs_pages_workspace_bytes(requests, pages)
        self.ws = torch.full((wsb,), 255, dtype=torch.uint8, device="cuda")
        self.pool = hs.make_page_pool(self.pools, requests, max_pages, pages, page_size, row_bytes, self.table, self.refs,
                                      self.free, self.count, self.ws, wsb, self.err)
        hs.hs_pages_init(self.pool)
        self.same()

    def same(self, flags=0):
        o = self.orc
        assert np.array_equal(self.table.cpu().numpy(), o.table)
        assert np.array_equal(self.refs.cpu().numpy(), o.refs)
        n = int(self.count.item())
        assert self.free.cpu().numpy()[:n].tolist() == o.free
        for raw, got, want in zip(self.raw, self.pools, o.pools):
            assert np.array_equal(got.cpu().numpy(), want)
            at = 256 + self.skew
            assert (raw[:at] == 0xA7).all() and (raw[at + want.size:] == 0xA7).all()
        assert int(self.err.item()) == flags
        self.err.zero_()
        o.check()

    def extend(self, r, a, b, stream=None):
        got = torch.full((len(r),), 55, dtype=torch.int32, device="cuda")
        self.hs.hs_pages_extend(self.pool, len(r), d(r), d(a), d(b), got, stream)
        want, flags = self.orc.extend(r, a, b)
        assert got.tolist() == want
        self.same(flags)
        return want

    def fork(self, p, c, n):
        got = torch.full((len(p),), 55, dtype=torch.int32, device="cuda")
        self.hs.hs_pages_fork(self.pool, len(p), d(p), d(c), d(n), got)
        want, flags = self.orc.fork(p, c, n)
        assert got.tolist() == want
        self.same(flags)
        return want

    def release(self, r, first=None, end=None):
        self.hs.hs_pages_free(self.pool, len(r), d(r), None if first is None else d(first), None if end is None else d(end))
        self.same(self.orc.release(r, first, end))

    def compact(self):
        self.hs.hs_pages_compact(self.pool)
        self.orc.compact()
        self.same()


@pytest.mark.parametrize("requests,max_pages,pages,page,row_bytes,layers,skew", [
    (1, 1, 1, 1, 1, 1, 0), (8, 12, 60, 16, 416, 2, 0), (8, 12, 60, 5, 656, 3, 0), (40, 9, 150, 4, 7, 1, 0),
    (40, 33, 700, 2, 20, 2, 4), (8, 12, 50, 16, 416, 1, 1), (300, 5, 1100, 1, 32, 8, 0), (64, 70, 3500, 3, 48, 1, 0)])
def test_random_runs_match_the_oracle(requests, max_pages, pages, page, row_bytes, layers, skew):
    """Sequences start, grow, branch, lose pages at either end, finish; the pool is packed now and then."""
    hs = _gpu()
    rng = np.random.default_rng(pages)
    s = Pair(hs, pages, requests, max_pages, pages, page, row_bytes, layers, skew)
    lens = np.zeros(requests, np.int64)
    most = max_pages * page
    for step in range(12):
        r = rng.permutation(requests)[:rng.integers(0, requests) + 1]
        new = np.minimum(lens[r] + rng.integers(0, 2 * most // 3 + 2, r.size), most)
        got = s.extend(r.tolist(), lens[r].tolist(), new.tolist())
        for x, w, n in zip(r, got, new):
            lens[x] = n if w >= 0 else lens[x]
        busy, idle = np.flatnonzero(lens > 0), np.flatnonzero(lens == 0)
        if busy.size and idle.size:
            c = rng.permutation(idle)[:rng.integers(0, idle.size) + 1]
            p = rng.choice(busy, c.size)
            n = np.array([rng.integers(0, lens[x] + 1) for x in p])
            got = s.fork(p.tolist(), c.tolist(), n.tolist())
            for x, w, k in zip(c, got, n):
                lens[x] = k if w >= 0 else 0
        if step % 2:
            gone = rng.permutation(requests)[:requests // 2 + 1]
            s.release(gone.tolist())
            lens[gone] = 0
        if step % 3 == 2:
            s.compact()
    s.release(list(range(requests)))
    s.compact()
    assert int(s.count.item()) == pages


def test_extend_refusals_and_padding():
    hs = _gpu()
    s = Pair(hs, 1, 6, 8, 12, 4)
    s.extend([0, -1, 6, 1, 1, 2, 3, 4, 5], [0, 0, 0, 0, 0, 5, -1, 0, 0], [9, 5, 4, 4, 8, 4, 4, 33, 0])
    s.extend([0, 2], [8, 0], [12, 4])  # index 2 of request 0 holds a page already
    s.extend([2, 3, 4, 5], [4, 0, 0, 0], [12, 32, 4, 0])  # 2 + 8 pages of 8, then a small entry after the one that does not fit
    s.extend([1], [0], [0])
    s.extend([5], [3, ], [4])  # within the page of tokens 0 .. 3: nothing to give


def test_fork_refusals_and_padding():
    hs = _gpu()
    s = Pair(hs, 2, 8, 8, 12, 4)
    s.extend([0, 1], [0, 0], [14, 8])
    s.fork([0, 0, -1, 0, 0, 8, 0, 0], [2, 2, 3, -1, 8, 3, 0, 1], [14] * 8)
    s.fork([0, 0, 0], [2, 3, 4], [33, -1, 0])
    s.fork([0, 0], [2, 3], [14, 13])
    s.fork([0, 1], [2, 4], [14, 8])  # request 2 holds pages by now
    s.fork([2, 0, 2, 1, 3], [5, 6, 7, 4, 0], [14, 14, 14, 14, 14])  # 0 holds pages and is a parent
    s.release([2])
    s.fork([1], [2], [14])  # longer than the parent's pages: the absent index stays absent


def test_free_ranges_repeats_and_padding():
    hs = _gpu()
    s = Pair(hs, 3, 6, 10, 40, 4)
    s.extend([0, 1, 2], [0, 0, 0], [40, 22, 7])
    s.fork([0, 1], [3, 4], [38, 22])
    s.release([0, -1, 6, 0, 3, 3], [2, 0, 0, 3, -5, 8], [5, 9, 9, 4, 2, 99])
    s.release([1, 1, 1])
    s.release([2], [9], [3])
    s.release([0, 1, 2, 3, 4, 5])
    s.release([5])


def test_compact_of_full_empty_and_packed_pools():
    hs = _gpu()
    s = Pair(hs, 4, 4, 40, 64, 8, 416, 4)
    s.compact()
    s.extend([0, 1, 2, 3], [0] * 4, [128, 128, 128, 128])
    s.compact()  # every page in use
    s.release([1])
    s.compact()
    s.compact()
    s.release([0, 2], [0, 5], [3, 11])
    s.compact()


def test_states_that_no_call_leaves_are_flagged_and_stay_in_bounds():
    """Counts, stack entries and table entries out of range: HS_FLAG_STATE, and no access outside
    (every index is checked before its use; the canaries stay)."""
    hs = _gpu()
    s = Pair(hs, 5, 4, 6, 10, 4)
    s.extend([0, 1], [0, 0], [10, 9])
    s.table[1, 1] = 10 ** 6
    s.table[1, 2] = -9
    got = torch.zeros(1, dtype=torch.int32, device="cuda")
    hs.hs_pages_fork(s.pool, 1, d([1]), d([2]), d([8]), got)
    assert s.err.item() == hs.HS_FLAG_STATE and s.table[2].tolist()[:3] == [3, -1, -1]
    s.err.zero_()
    hs.hs_pages_fork(s.pool, 1, d([1]), d([3]), d([7]), got)
    assert s.err.item() == hs.HS_FLAG_STATE and got.item() == -1 and (s.table[3] == -1).all()
    s.err.zero_()
    hs.hs_pages_compact(s.pool)
    assert s.err.item() == hs.HS_FLAG_STATE
    s.err.zero_()
    hs.hs_pages_free(s.pool, 1, d([1]))
    assert s.err.item() == hs.HS_FLAG_STATE and (s.table[1] == -1).all()
    s.err.zero_()
    s.count.fill_(10 ** 6)
    s.free.fill_(-3)
    hs.hs_pages_extend(s.pool, 1, d([1]), d([0]), d([9]), got)
    assert s.err.item() == hs.HS_FLAG_STATE and (s.table[1] == -1).all()
    for raw in s.raw:
        assert (raw[:256] == 0xA7).all() and (raw[-256:] == 0xA7).all()


def test_a_step_replayed_from_a_graph():
    hs = _gpu()
    s = Pair(hs, 6, 16, 40, 300, 8, 416, 2)
    s.extend(list(range(4)), [0] * 4, [90, 64, 33, 200])
    state = [s.table, s.refs, s.free, s.count]
    before = [x.clone() for x in state]
    args = d([0, 1, 2, 3]), d([90, 64, 33, 200]), d([97, 65, 40, 300]), d([0, 1, 2, 3]), d([4, 5, 6, 7]), d([97, 65, 40, 300]), d([1, 4])

    def step(st):
        hs.hs_pages_extend(s.pool, 4, *args[:3], None, st)
        hs.hs_pages_fork(s.pool, 4, *args[3:6], None, st)
        hs.hs_pages_free(s.pool, 2, args[6], None, None, st)
        hs.hs_pages_compact(s.pool, st)

    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        step(st)
    orc = s.orc
    orc.extend([0, 1, 2, 3], [90, 64, 33, 200], [97, 65, 40, 300])
    orc.fork([0, 1, 2, 3], [4, 5, 6, 7], [97, 65, 40, 300])
    orc.release([1, 4])
    orc.compact()
    first = [p.clone() for p in s.pools]
    for _ in range(2):
        for x, y in zip(state + s.pools, before + first):
            x.copy_(y)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        s.same()


def test_a_generation_with_4_bit_rows_from_first_token_to_last():
    """As a server uses them: pages are taken, prompts' rows written, a window query and a top-k query
    read them, sequences branch and go on apart, some finish, the pool is packed, and the rest reads on."""
    hs = _gpu()
    import test_gpu_fp4 as T
    rng = np.random.default_rng(12)
    R, mp, ps, H, g = 6, 20, 16, 24, 0.5
    s = Pair(hs, 7, R, mp, 80, ps)
    pool, total = s.pools[0], 80 * ps
    history = {}  # request -> its tokens' bf16 bits

    def write(r, new):
        start = len(history.get(r, ()))
        history[r] = np.concatenate((history[r], new)) if start else new
        t = np.arange(start, len(history[r]))
        rows = s.orc.table[r, t // ps] * ps + t % ps
        hs.hs_fp4_pack_rows(len(t), T.d(new), 576, d(rows), g, pool, total, s.err)
        s.orc.pools[0][rows] = F.pack(new, g)

    def grow(rs, ks):
        old = [len(history.get(r, ())) for r in rs]
        s.extend(rs, old, [a + k for a, k in zip(old, ks)])
        for r, k in zip(rs, ks):
            write(r, T.tokens(rng, k))
        s.same()

    def read():
        lens = np.array([len(history.get(r, ())) for r in range(R)], np.int32)
        q = T.bf16_bits(rng.standard_normal((R, 2, H, 576)))
        o, lse, err = T.window(hs, q, pool, ps, lens, s.table.cpu().numpy(), 40, 3, g, 2)
        assert err == 0
        for r in range(R):
            rec = F.pack(history[r], g) if r in history else np.zeros((0, 416), np.uint8)
            for i in range(2):
                t = F.window_tokens(int(lens[r]) - 2 + i, 40, 3)
                T.check(q[r, i], rec[t], g, o[r, i], lse[r, i], f"window: request {r} query {i}")
        top = np.full((R, 30), -1, np.int32)
        picks = {}
        for r in history:
            t = picks[r] = rng.permutation(len(history[r]))[:30]
            top[r, :len(t)] = s.orc.table[r, t // ps] * ps + t % ps
        o, lse, err = T.sparse(hs, q[:, 0].copy(), pool, d(top), g, 1)
        assert err == 0
        for r in history:
            T.check(q[r, 0], F.pack(history[r], g)[picks[r]], g, o[r], lse[r], f"top-k: request {r}")

    grow([0, 1, 2], [100, 47, 1])
    read()
    n = [len(history[0]), 40]
    s.fork([0, 1], [3, 4], n)
    history[3], history[4] = history[0][:n[0]].copy(), history[1][:n[1]].copy()
    read()
    for _ in range(3):
        grow([0, 1, 2, 3, 4], [1, 2, 20, 7, 1])
        read()
    for r in (0, 2):
        s.release([r])
        del history[r]
    s.compact()
    read()
    grow([1, 3, 4, 0], [30, 1, 12, 65])
    read()
    back = d(s.orc.table[4, 0] * ps + np.arange(16))
    out = torch.zeros(16, 576, dtype=torch.int16, device="cuda")
    hs.hs_fp4_unpack_rows(16, pool, total, back, g, out, 576, s.err)
    lat, rope = F.unpack(F.pack(history[4][:16], g), g)
    assert np.array_equal(F.bf16_decode(out.cpu().numpy().view(np.uint16)), np.concatenate((lat, rope), 1))


def test_a_4_bit_pool_through_the_resolver():
    """row_bytes 416 through hs_create, hs_resolve and hs_backup, its rows read by the 4-bit attention."""
    hs = _gpu()
    import test_gpu_fp4 as T
    R, K, H, ctx = 3, 24, 32, 400
    rng = np.random.default_rng(5)
    kv = {(r, t): T.tokens(rng, 1) for r in range(R) for t in range(ctx)}
    cfg = hs.make_config(R, K, H, 416, 1, 0, ctx, 0)
    host = np.zeros((R * ctx, 416), np.uint8)
    for (r, t), x in kv.items():
        host[r * ctx + t] = F.pack(x, 1.0)[0]
    host_t = torch.from_numpy(host).pin_memory()
    dev = torch.zeros(R * (H + 1), 416, dtype=torch.uint8, device="cuda")
    ws = torch.zeros(hs.hs_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    h = hs.hs_create(cfg, [host_t], [dev], R * ctx, R * (H + 1), ws)
    lens = d([300, 350, 399])
    hcl = torch.arange(R * ctx, dtype=torch.int32, device="cuda").view(R, ctx)
    dbl = torch.arange(R * (H + 1), dtype=torch.int32, device="cuda").view(R, H + 1)
    tok, st = torch.full((R, H), -1, dtype=torch.int32, device="cuda"), torch.zeros(R, H, dtype=torch.int32, device="cuda")
    clk, out = torch.zeros(R, dtype=torch.int32, device="cuda"), torch.zeros(R, K, dtype=torch.int32, device="cuda")
    # the newest tokens' rows: written where the resolver looks for them, then backed up
    newest = np.concatenate([T.tokens(rng, 1) for _ in range(R)])
    err = T.flags()
    hs.hs_fp4_pack_rows(R, T.d(newest), 576, dbl[:, H].contiguous(), 1.0, dev, R * (H + 1), err)
    top = np.stack([np.concatenate(([n - 1], rng.permutation(n - 1)[:K - 1])) for n in (300, 350, 399)]).astype(np.int32)
    hs.hs_resolve(h, R, d(top), lens, hcl, dbl, tok, st, clk, None, out, None)
    hs.hs_backup(h, R, lens, hcl, dbl, None)
    torch.cuda.synchronize()
    assert hs.hs_get_error(h) == 0 and int(err.item()) == 0
    q = T.bf16_bits(rng.standard_normal((R, 16, 576)))
    o, lse, e = T.sparse(hs, q, dev, out, 1.0, 2)
    assert e == 0
    for r in range(R):
        n = (300, 350, 399)[r]
        rec = np.concatenate([F.pack(newest[r:r + 1] if t == n - 1 else kv[r, int(t)], 1.0) for t in top[r]])
        T.check(q[r], rec, 1.0, o[r], lse[r], f"request {r}")
        assert np.array_equal(host_t.numpy()[r * ctx + n - 1], F.pack(newest[r:r + 1], 1.0)[0])
    hs.hs_destroy(h)
