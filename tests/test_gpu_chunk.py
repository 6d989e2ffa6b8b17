"""GPU parity of hs_chunk_mla against the oracle in 64 bits.

Per output element, with A_i = sum_j p_j |latent_ji|, B = max_j |sm| sum_d |q_d k_jd| of the head and C_i = sum_j
|latent_ji| over the rows that it sees:
* q goes through f16, over a power of two where the head's largest is below 1 or above 65504: off by up to 2^-25 of the
  head's largest, and only where a value is below 2^-14 of it; under 2^-16 of B for heads and rows whose values are of like
  sizes, as here;
* latents go through f16: exact where the scale is a power of two (4 bits of code), else off by 2^-11 of themselves, and
  by 2^-25 where they are under 2^-14: r = 2^-11 of each, and nothing for powers of two. RoPE values of 8 bits: exact
  but for those under 2^-14, off by up to 2^-25 (their products are under 2^-16 of B);
* scores: products of 11-bit values are exact in the accumulator; 36 accumulations of 16 products each round (or cut) by
  at most 2^-22 of sum |q_d k_d|: with q's and RoPE's shares E = (2^-16 + 2 r) B (r for the latent, twice for safety of
  none: sum |q| |latent| is part of B);
* weights: exp of a score that is off by E is off by E relative, 2 E after normalising (first order: E < 0.1 here); a
  weight rounded to f16 is off by 2^-11 of itself, and by 2^-32 of the largest of its part of the sequence where it is
  smaller than 2^-21 of that;
* values: r of each;  sums and the join of parts in 32 bits: 2^-16;  the bf16 result: 2^-8 |o_i|;
    |d o_i| <= (2 E + 2^-11 + r + 2^-16) A_i + 2^-32 C_i + 2^-8 |o_i|
* lse: |d| <= E + 2^-20 (1 + |lse|).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import chunk as C  # noqa: E402
from oracle.sparse_mla import bf16_decode  # noqa: E402

pytestmark = pytest.mark.gpu
SM = 0.0722


def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hierarchical_sparse_attention_gb300 as hs
    return hs


def bits(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def d(x):
    x = np.ascontiguousarray(x)
    return torch.from_numpy(x.view(np.int16) if x.dtype == np.uint16 else x).cuda()


def make_pool(rng, rows, any_scale=False, size=1.0):
    kv = rng.standard_normal((rows, 576)) * size
    kv[:, :512:37] *= 6
    kv[:, 5:512:11] *= 0.05
    rec = np.empty((rows, 656), np.uint8)
    rec[:, :528], rope = C.pack(bits(kv))
    if any_scale:
        rec[:, 512:528] = (rec[:, 512:528].copy().view(np.float32) * rng.uniform(0.5, 1, (rows, 4)).astype(np.float32)).view(np.uint8)
    rec[:, 528:] = bits(rope).view(np.uint8)
    return rec


class Batch:
    """Entries (tokens with the new ones, new ones) of a call, with random pages of a pool that has room for them."""

    def __init__(self, rng, heads, entries, page, room=0, any_scale=False, size=1.0, q_size=1.0, spare=3):
        self.heads, self.page = heads, page
        self.lens = np.array([e[0] for e in entries], np.int32)
        self.count = np.array([e[1] for e in entries], np.int64)
        self.offsets = np.concatenate(([0], np.cumsum(self.count))).astype(np.int32)
        self.max_tokens = int(self.offsets[-1]) + room
        held = -(-np.maximum(self.lens, 0).astype(np.int64) // page)
        self.max_blocks = int(max(1, held.max())) + 1
        pages = int(held.sum()) + spare
        self.tables = np.full((len(entries), self.max_blocks), -1, np.int32)
        perm, at = rng.permutation(pages).astype(np.int32), 0
        for i, h in enumerate(held):
            self.tables[i, :h] = perm[at:at + h]
            at += int(h)
        self.pool = make_pool(rng, pages * page, any_scale, size)
        self.q = bits(rng.standard_normal((max(1, self.max_tokens), heads, 576)) * q_size)
        self.r = 2.0 ** -11 if any_scale else 0.0
        self.kv_room = int((-(-np.maximum(self.lens, 0).astype(np.int64) // 64) * 64)[self.count > 0].sum())
        self.sm = SM

    def upload(self):
        self.dev = {k: d(getattr(self, k)) for k in ("offsets", "lens", "q", "pool", "tables")}
        return self

    def call(self, hs, kv_room=None, fill=0.0, ws=None, stream=None):
        if not hasattr(self, "dev"):
            self.upload()
        t, h = self.max_tokens, self.heads
        kv_room = self.kv_room if kv_room is None else kv_room
        n = len(self.lens)
        nbytes = hs.hs_chunk_mla_workspace_bytes(n, h, t, kv_room)
        if ws is None:
            ws = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda")
        o = torch.full((max(1, t), h, 512), fill, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((max(1, t), h), fill, dtype=torch.float32, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        x = self.dev
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        hs.hs_chunk_mla(n, h, t, x["offsets"], x["lens"], x["q"], x["pool"], self.pool.shape[0], self.page, self.max_blocks, x["tables"], self.sm, o, lse, kv_room, ws, nbytes, err,
                        stream)
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        return o, lse, err

    def expected(self, i, lens=None):
        a, b = int(self.offsets[i]), int(self.offsets[i + 1])
        return C.chunk_entry(bf16_decode(self.q[a:b]), int(self.lens[i]), b - a, self.tables[i], self.page, self.pool, self.sm)

    def check(self, o, lse, entries=None):
        o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
        for i in range(len(self.lens)) if entries is None else entries:
            a, b = int(self.offsets[i]), int(self.offsets[i + 1])
            if a == b:
                continue
            want, wl, A, B, Cs = self.expected(i)
            E = (2.0 ** -16 + 2 * self.r) * B
            assert E.max() < 0.1
            bound = (2 * E[..., None] + 2.0 ** -11 + self.r + 2.0 ** -16) * A + 2.0 ** -32 * Cs + 2.0 ** -8 * np.abs(want)
            off = np.abs(o[a:b] - want)
            assert (off <= bound).all(), f"entry {i}: {np.nanmax(off / np.maximum(bound, 1e-300))} of the bound"
            none = np.isinf(wl)
            assert np.array_equal(lse[a:b][none], wl[none])
            assert (np.abs(lse[a:b] - wl)[~none] <= (E + 2.0 ** -20 * (1 + np.abs(wl)))[~none]).all(), f"entry {i}: lse"


SHAPES = [
    (16, 64, [(1, 1)]), (1, 64, [(5, 5)]), (16, 64, [(64, 1), (65, 1), (63, 2), (128, 3), (129, 4)]), (128, 64, [(200, 3), (64, 64)]), (128, 16, [(300, 1)]),
    (64, 48, [(100, 2), (77, 77), (500, 5)]), (65, 1, [(130, 2), (3, 3)]), (127, 7, [(90, 2)]), (3, 128, [(257, 100), (1, 1)]), (40, 64, [(190, 7)]), (2, 5, [(333, 200)]),
    (1, 16, [(700, 300), (10, 1)]), (16, 64, [(1000, 1), (0, 0), (2000, 17), (64, 64), (0, 0), (31, 8)]), (128, 64, [(777, 1)] * 5 + [(130, 60)]), (100, 3, [(50, 20), (49, 1)]),
    (16, 64, [(8192, 1), (101, 1)]), (32, 64, [(5000, 4)] * 3),
]


@pytest.mark.parametrize("any_scale", [False, True])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_shapes(shape, any_scale):
    hs = _gpu()
    heads, page, entries = SHAPES[shape]
    b = Batch(np.random.default_rng(shape), heads, entries, page, any_scale=any_scale)
    o, lse, err = b.call(hs)
    b.check(o, lse)
    assert int(err.item()) == 0


def test_rows_behind_the_last_token_and_between_entries_stay():
    hs = _gpu()
    b = Batch(np.random.default_rng(40), 16, [(70, 3), (0, 0), (9, 2)], 64, room=30)
    o, lse, err = b.call(hs, fill=7.0)
    b.check(o, lse)
    assert (o[5:] == 7).all() and (lse[5:] == 7).all() and int(err.item()) == 0


def test_queries_that_see_nothing():
    """More queries than tokens (the first stand before the sequence), an empty sequence, pages that are not there, alone
    and among others, and rows past the pool."""
    hs = _gpu()
    b = Batch(np.random.default_rng(41), 16, [(3, 7), (0, 2), (150, 4), (200, 3), (70, 70)], 16)
    b.tables[2] = -1
    b.tables[3, 2:5] = [-1, -5, 2 ** 31 - 1]
    b.tables[3, 12] = b.pool.shape[0] // 16 - 1
    b.tables[4, 0] = -1  # the first 16 queries see nothing
    b.pool = b.pool[:-9]  # (the pool's last page ends early)
    o, lse, err = b.call(hs, fill=3.0)
    b.check(o, lse)
    assert (o[:4] == 0).all() and (lse[7:9] == -np.inf).all() and int(err.item()) == hs.HS_FLAG_DEVROW


def test_bad_lengths_and_offsets():
    hs = _gpu()
    b = Batch(np.random.default_rng(42), 16, [(70, 3), (80, 2), (90, 4), (50, 1)], 64, room=6)
    good = b.lens.copy()
    for bad in (-1, b.max_blocks * 64 + 1, 2 ** 31 - 1):
        b.lens = good.copy()
        b.lens[1] = bad
        b.upload()
        o, lse, err = b.call(hs, fill=2.0, kv_room=1024)
        assert int(err.item()) == hs.HS_FLAG_SEQLEN and (o[3:5] == 0).all() and (lse[3:5] == -np.inf).all()
        b.check(o, lse, [0, 2, 3])
    b.lens = good
    b.upload()
    # (in the second case entry 2 takes tokens of entry 0 too: what both write is either's)
    for at, value, keep in ((1, -4, [2, 3]), (2, 1, [3]), (4, b.max_tokens + 1, [0, 1, 2])):
        off = b.offsets.copy()
        off[at] = value
        b.dev["offsets"] = d(off)
        o, lse, err = b.call(hs, fill=2.0, kv_room=1024)
        assert int(err.item()) == hs.HS_FLAG_SEQLEN
        b.check(o, lse, keep)
        assert (o[10:] == 2).all()


def test_sequences_that_do_not_fit():
    hs = _gpu()
    b = Batch(np.random.default_rng(43), 16, [(70, 3), (0, 1), (300, 2), (10, 1), (0, 1), (64, 0)], 64)
    for room, fit in ((128 + 320 + 64, 4), (128 + 320 + 63 // 64 * 64, 3), (128 + 256, 2), (128, 2), (64, 0), (0, 0)):
        o, lse, err = b.call(hs, kv_room=room, fill=5.0)
        assert int(err.item()) == (0 if fit == 4 else hs.HS_FLAG_FULL)
        for i in range(6):
            if i in (1, 4) or i >= fit:
                a, e = int(b.offsets[i]), int(b.offsets[i + 1])
                assert (o[a:e] == 0).all() and (lse[a:e] == -np.inf).all()
            else:
                b.check(o, lse, [i])


def test_nan_rows_reach_only_the_queries_that_see_them():
    hs = _gpu()
    b = Batch(np.random.default_rng(44), 16, [(100, 40), (80, 5)], 64)
    at = int(b.tables[0, 1]) * 64 + 80 - 64  # token 80 of the first sequence, seen from query 20 on
    b.pool[at, 512:516] = np.array([np.nan], np.float32).view(np.uint8)
    b.pool[int(b.tables[1, 0]) * 64 + 3, 7] = 0x7F  # a NaN code, seen by all of the second's
    unused = np.setdiff1d(np.arange(b.pool.shape[0] // 64), b.tables)
    b.pool[unused * 64, 512:528] = 0xFF  # rows of no sequence
    b.pool[int(b.tables[0, 1]) * 64 + 50, 512:528] = 0xFF  # behind the sequence's end, on its last page
    o, lse, err = b.call(hs)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(o[:20]).all() and np.isnan(lse[20:45]).all() and np.isnan(o[20:40]).all(-1).all()
    assert np.isnan(o[40:45]).any(-1).all() and int(err.item()) == 0
    want = b.expected(0)
    assert (np.abs(o[:20] - want[0][:20]) <= 2.0 ** -7 * (np.abs(want[0][:20]) + want[2][:20])).all()


def test_rope_values_that_are_not_finite():
    hs = _gpu()
    for value in (0x7FC0, 0x7F80, 0xFF80):
        b = Batch(np.random.default_rng(45), 16, [(100, 40)], 64)
        b.pool[int(b.tables[0, 1]) * 64 + 80 - 64, 528:530] = np.array([value], np.uint16).view(np.uint8)
        o, lse, _ = b.call(hs)
        assert torch.isfinite(o[:20].float()).all() and torch.isfinite(lse[:20]).all()
        if value == 0x7FC0:
            assert torch.isnan(lse[20:]).all()


@pytest.mark.parametrize("q_size,size", [(2.0 ** 60, 2.0 ** -70), (2.0 ** -60, 2.0 ** 8), (2.0 ** 100, 2.0 ** -100), (300.0, 1.0), (30.0, 8.0)])
def test_sizes_of_queries_and_rows(q_size, size):
    """The scale brings the scores to a spread of about 2, whatever q's size; rows' sizes within what f16 holds."""
    hs = _gpu()
    size = max(size, 2.0 ** -6)
    b = Batch(np.random.default_rng(46), 40, [(200, 9), (64, 2)], 64, size=size, q_size=q_size)
    b.sm = float(np.float32(0.0722 / (q_size * size) * 2))
    o, lse, err = b.call(hs)
    b.check(o, lse)


def test_heads_of_very_different_sizes_and_zero_queries():
    hs = _gpu()
    b = Batch(np.random.default_rng(47), 8, [(150, 20)], 64)
    q = bf16_decode(b.q)
    q[:, 1] = 0
    q[:, 2] *= 2.0 ** -40
    q[:, 3] *= 2.0 ** -100
    b.q = bits(q)
    o, lse, _ = b.call(hs)
    b.check(o, lse)


@pytest.mark.parametrize("sm", [0.0, -0.0722, 1e-30])
def test_scales_of_other_signs(sm):
    hs = _gpu()
    b = Batch(np.random.default_rng(48), 16, [(300, 5), (20, 20)], 64)
    b.sm = sm
    o, lse, _ = b.call(hs)
    b.check(o, lse)


def test_one_row_outweighs_the_others():
    """Scores of hundreds: weights underflow but for one row's, on either side of where the sequence is cut in parts; a
    maximum that rises block by block."""
    hs = _gpu()
    rng = np.random.default_rng(49)
    b = Batch(rng, 16, [(3000, 6), (700, 1)], 64)
    lat, rope = C.unpack(b.pool)
    for i, t in ((0, 2100), (1, 10)):
        row = int(b.tables[i, t // 64]) * 64 + t % 64
        a, e = int(b.offsets[i]), int(b.offsets[i + 1])
        b.q[a:e, 3] = bits(np.concatenate((lat[row], rope[row])) * 4)
    for t in range(0, 3000, 64):  # rising
        row = int(b.tables[0, t // 64]) * 64 + t % 64
        b.pool[row, 528:] = bits(np.full(64, t / 300.0)).view(np.uint8)
    b.q[2, 5, 512:] = bits(np.full(64, 1.0))
    o, lse, _ = b.call(hs)
    b.check(o, lse)


def test_parts_of_long_sequences():
    """One sequence over many CTA pairs; several, whose parts end everywhere; the join of parts of few heads."""
    hs = _gpu()
    for heads, entries, page in ((16, [(20000, 2)], 64), (128, [(3000, 1), (5000, 2), (64, 1), (1, 1), (4100, 3)], 64), (5, [(9000, 30), (12000, 1)], 16)):
        b = Batch(np.random.default_rng(50 + heads), heads, entries, page)
        o, lse, err = b.call(hs)
        b.check(o, lse)
        again = b.call(hs)
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1]) and int(err.item()) == 0


def test_more_tiles_than_pairs():
    hs = _gpu()
    b = Batch(np.random.default_rng(51), 128, [(90 + i, 1 + i % 3) for i in range(120)], 64)
    o, lse, _ = b.call(hs)
    b.check(o, lse, range(0, 120, 7))
    b = Batch(np.random.default_rng(52), 16, [(65 * i % 400 + 1, min(65 * i % 400 + 1, 5)) for i in range(1300)], 64)
    o, lse, _ = b.call(hs)
    b.check(o, lse, range(0, 1300, 29))


def test_many_entries_few_of_them_with_tokens():
    """More entries than one CTA of the kernels looks over at once, and few with queries; with and without room for all."""
    hs = _gpu()
    rng = np.random.default_rng(58)
    for n in (1024, 1025, 5000):
        entries = [(0, 0)] * n
        for i in rng.permutation(n)[:25]:
            entries[i] = (int(rng.integers(1, 700)), 1)
        entries[n - 1], entries[0] = (130, 3), (65, 2)
        entries = [(s, min(q, s)) for s, q in entries]
        b = Batch(rng, 16, entries, 64)
        o, lse, err = b.call(hs)
        b.check(o, lse)
        assert int(err.item()) == 0
        o, lse, err = b.call(hs, kv_room=b.kv_room + 64 * 50)
        b.check(o, lse)
        o, lse, err = b.call(hs, kv_room=b.kv_room - 64)  # all but the last one
        b.check(o, lse, [i for i in range(n - 1) if b.count[i]])
        assert (lse[-3:] == -np.inf).all() and int(err.item()) == hs.HS_FLAG_FULL


def test_sequences_around_the_shortest_that_is_cut():
    """Seven, eight and nine blocks: below eight nothing is cut, and no join is launched where the sizes allow none."""
    hs = _gpu()
    for seq in (447, 448, 449, 511, 512, 513, 577):
        b = Batch(np.random.default_rng(seq), 128, [(seq, 1)], 64)
        b.max_blocks = -(-seq // 64)
        b.tables = np.ascontiguousarray(b.tables[:, :b.max_blocks])
        o, lse, err = b.call(hs)
        b.check(o, lse)
        b = Batch(np.random.default_rng(seq), 16, [(seq, 9), (seq - 3, 1)], 1)
        o, lse, err = b.call(hs)
        b.check(o, lse)


def test_captured_and_replayed_with_other_lengths_and_two_graphs_of_one_workspace():
    hs = _gpu()
    rng = np.random.default_rng(53)
    a = Batch(rng, 16, [(300, 10), (500, 1), (64, 4)], 64, room=20).upload()
    room = 64 * 40
    n, t = 3, a.max_tokens
    nbytes = hs.hs_chunk_mla_workspace_bytes(n, 16, t, room)
    ws = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    outs, graphs = [], []
    for _ in range(2):
        o = torch.zeros(t, 16, 512, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros(t, 16, dtype=torch.float32, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=side):
            x = a.dev
            hs.hs_chunk_mla(n, 16, t, x["offsets"], x["lens"], x["q"], x["pool"], a.pool.shape[0], 64, a.max_blocks, x["tables"], a.sm, o, lse, room, ws, nbytes, err, side)
        outs.append((o, lse))
        graphs.append(g)
    lens, count = a.lens.copy(), a.count.copy()
    for new in ([(300, 10), (500, 1), (64, 4)], [(290, 1), (0, 0), (64, 30)], [(64, 2), (500, 8), (1, 1)]):
        a.lens = np.array([x[0] for x in new], np.int32)
        a.offsets = np.concatenate(([0], np.cumsum([x[1] for x in new]))).astype(np.int32)
        a.dev["lens"].copy_(d(a.lens))
        a.dev["offsets"].copy_(d(a.offsets))
        for g, (o, lse) in zip(graphs, outs):
            o.fill_(9)
            g.replay()
            g.replay()
            a.check(o, lse)
            assert (o[int(a.offsets[-1]):] == 9).all()


def test_two_streams_at_once_with_workspaces_of_their_own():
    hs = _gpu()
    b = [Batch(np.random.default_rng(54 + i), 64, [(2000, 8), (900 + i, 3)], 64).upload() for i in range(2)]
    alone = [x.call(hs) for x in b]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in b]
    for _ in range(5):
        got = [x.call(hs, stream=s) for x, s in zip(b, streams)]
        torch.cuda.synchronize()
        for (o, lse, err), (o0, l0, _) in zip(got, alone):
            assert torch.equal(o, o0) and torch.equal(lse, l0) and int(err.item()) == 0
    b[0].check(*alone[0][:2])


def test_a_pool_past_four_gigabytes():
    hs = _gpu()
    rng = np.random.default_rng(56)
    b = Batch(rng, 16, [(200, 5), (130, 1)], 64)
    pages = 7_000_000 // 64
    big = torch.empty(pages * 64, 656, dtype=torch.uint8, device="cuda")
    far = rng.permutation(pages - 8)[:b.pool.shape[0] // 64].astype(np.int64)
    far[:4] = pages - 1 - np.arange(4)
    old = b.pool.reshape(-1, 64, 656)
    big.view(-1, 64, 656)[d(far)] = d(old)
    held = b.tables >= 0
    tables = b.tables.copy()
    tables[held] = far[b.tables[held]]
    b.upload()
    b.dev["pool"], b.dev["tables"] = big, d(tables.astype(np.int32))
    small = b.pool
    b.pool = np.broadcast_to(small[:1], (pages * 64, 656))  # (the call takes its number of rows from here)
    o, lse, err = b.call(hs)
    b.pool = small
    b.check(o, lse)
    assert int(err.item()) == 0


def test_a_step_from_pages_to_attention():
    """Pages are given, the batch planned, rows written, attended, twice: a first chunk and then verify steps, as a server
    does it; the second sequence is a fork of the first."""
    hs = _gpu()
    rng = np.random.default_rng(57)
    slots, max_pages, page, heads = 5, 8, 16, 16
    num_pages = 30
    pool = torch.zeros(num_pages * page, 656, dtype=torch.uint8, device="cuda")
    ints = lambda *s: torch.full(s, -9, dtype=torch.int32, device="cuda")  # noqa: E731
    table, refs, free, count, err = ints(slots, max_pages), ints(num_pages), ints(num_pages), ints(1), torch.zeros(1, dtype=torch.int32, device="cuda")
    wsb = hs.hs_pages_workspace_bytes(slots, num_pages)
    pp = hs.make_page_pool([pool], slots, max_pages, num_pages, page, 656, table, refs, free, count, torch.zeros(wsb, dtype=torch.uint8, device="cuda"), wsb, err)
    hs.hs_pages_init(pp)
    w = bits(1 + 0.1 * rng.standard_normal(512))
    ang = np.arange(200)[:, None] * 10000.0 ** (-np.arange(0, 64, 2) / 64.0)
    rope = np.concatenate((np.cos(ang), np.sin(ang)), 1).astype(np.float32)
    kept = {}  # of a request: its tokens' rows, as the oracle writes them

    def step(req, old, new, room):
        n = len(req)
        r, o_, n_ = (d(np.array(x, np.int32)) for x in (req, old, new))
        hs.hs_pages_extend(pp, n, r, o_, n_)
        off, lens, ent, pos, rows, tabs = ints(n + 1), ints(n), ints(room), ints(room), ints(room), ints(n, max_pages)
        hs.hs_batch_plan(n, r, o_, n_, slots, table, max_pages, page, num_pages * page, room, off, lens, ent, pos, rows, max_pages, tabs, err)
        kv = bits(rng.standard_normal((room, 576)))
        hs.hs_fp8_pack_rows(room, d(kv), 576, rows, d(w), 1e-6, pos, d(rope), 200, pool, num_pages * page, err)
        q = bits(rng.standard_normal((room, heads, 576)))
        kv_room = 64 * 2 * n
        nbytes = hs.hs_chunk_mla_workspace_bytes(n, heads, room, kv_room)
        o = torch.zeros(room, heads, 512, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros(room, heads, device="cuda")
        hs.hs_chunk_mla(n, heads, room, off, lens, d(q), pool, num_pages * page, page, max_pages, tabs, SM, o, lse, kv_room,
                        torch.zeros(nbytes, dtype=torch.uint8, device="cuda"), nbytes, err)
        at = 0
        for i, x in enumerate(req):
            if x < 0:
                continue
            m = new[i] - old[i]
            rec, rp = C.pack(kv[at:at + m], w, 1e-6, np.arange(old[i], new[i]), rope)
            kept[x] = kept.get(x, [])[:old[i]] + list(np.concatenate((rec, bits(rp).view(np.uint8)), 1))
            b = Batch.__new__(Batch)
            b.heads, b.page, b.pool, b.sm, b.r = heads, 1, np.array(kept[x]), SM, 2.0 ** -16  # (r: a rotated value may fall to the other side)
            b.lens, b.offsets = np.array([new[i]], np.int32), np.array([0, m], np.int32)
            b.tables, b.q = np.arange(new[i], dtype=np.int32)[None], q[at:at + m]
            b.check(o[at:at + m], lse[at:at + m])
            at += m
        assert (o[at:] == 0).all() and int(err.item()) == 0

    step([3, -1], [0, 0], [37, 4], 40)
    hs.hs_pages_fork(pp, 1, d(np.array([3], np.int32)), d(np.array([1], np.int32)), d(np.array([37], np.int32)))
    kept[1] = list(kept[3])
    step([1, 0, 3], [37, 0, 37], [41, 20, 38], 30)
    step([0, 1, 3], [20, 41, 38], [21, 42, 39], 3)
