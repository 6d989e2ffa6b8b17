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


def loud(rng, n, top):
    """n rows whose RoPE values make scores of any sign up to about top^2 x 64, and their latents."""
    kv = rng.standard_normal((n, 576))
    kv[:, 512:] = rng.choice([-1.0, 1.0], (n, 64)) * top * rng.uniform(0.25, 1, (n, 64))
    return F.pack(T.bf16_bits(kv), 1.0)


@pytest.mark.parametrize("top", [2.0 ** 4, 2.0 ** 9, 2.0 ** 12, 2.0 ** 15, 2.0 ** 25])
@pytest.mark.parametrize("sm", [T.SM, -1.0])
@pytest.mark.parametrize("splits", [1, 3])
def test_scores_of_any_size_average_the_rows(top, sm, splits):
    """A score passes 2^28 where its rounding in 32 bits is whole powers of two of a weight. Whatever the scores
    are off by (test_gpu_fp4's E), weights are positive and add up to one:
    * of a single row the weight is exactly 1: o is its latent, off by the bf16 rounding, 2^-9 of it;
    * of many rows, a weight is off by 2^-11 of itself by its rounding, and by 2^-25 of the largest: o lies between the
      rows' least and largest latents, but for 2^-11 + 2^-16 (sums) + 2^-9 (bf16) < 2^-8 and n 2^-25 of the largest
      magnitude."""
    hs = T._gpu()
    rng = np.random.default_rng(int(np.log2(top)))
    pool = loud(rng, 400, top)
    q = rng.standard_normal((6, 24, 576))
    q[:, :, 512:] = rng.choice([-1.0, 1.0], (6, 24, 64)) * top * rng.uniform(0.25, 1, (6, 24, 64))
    q = T.bf16_bits(q)
    rows = np.full((6, 200), -1, np.int32)
    rows[0, 0], rows[1, 199], rows[2, 70] = 3, 5, 8  # one row only
    rows[3:] = rng.integers(0, 400, (3, 200))
    rows[5, 3:] = rows[5, 0]  # three rows, one of them again and again
    o, lse, err = T.sparse(hs, q, T.d(pool), T.d(rows), 1.0, splits, sm)
    assert err == 0
    lat, rope = F.unpack(pool, 1.0)
    for r in range(6):
        mine = rows[r][rows[r] >= 0]
        if r < 3:
            assert (np.abs(o[r] - lat[mine]) <= 2.0 ** -9 * np.abs(lat[mine])).all()
        low, high = lat[mine].min(0), lat[mine].max(0)
        slack = (2.0 ** -8 + mine.size * 2.0 ** -25) * np.abs(lat[mine]).max(0)
        assert (o[r] >= low - slack).all() and (o[r] <= high + slack).all()
        _, want, _, B = F.attend(T.bf16_decode(q[r]), lat[mine], rope[mine], sm)
        assert (np.abs(lse[r] - want) <= 2.0 ** -16 * B + 2.0 ** -20 * (1 + np.abs(want))).all()


@pytest.mark.parametrize("order", [1, -1])
def test_one_score_far_above_all_others_takes_all(order):
    """Scores 2^23 k for k = 0 .. 15, all of them exact (one RoPE value, powers of two times k) and so far apart that a
    rounding does not move a weight off 0 or 1: every query sees the loudest row alone, rows rising or falling."""
    hs = T._gpu()
    rng = np.random.default_rng(5)
    kv = np.zeros((16, 576))
    kv[:, :512] = rng.standard_normal((16, 512))
    kv[:, 512] = 2.0 ** 13 * np.arange(16)
    rec = F.pack(T.bf16_bits(kv), 1.0)[::order].copy()
    pool = np.repeat(rec, 60, 0)
    q = np.zeros((1, 20, 576))
    q[:, :, 512] = 2.0 ** 14
    rows = np.arange(16 * 60, dtype=np.int32)[None]
    o, lse, err = T.sparse(hs, T.bf16_bits(q), T.d(pool), T.d(rows), 1.0, 1, 2.0 ** -4)
    lat, _ = F.unpack(rec, 1.0)
    top = lat[15 if order > 0 else 0]
    assert err == 0
    # sixty equal rows' weights are 1 / 60 each: their sum in 32 bits is off by 2^-24 of it a term
    assert (np.abs(o[0] - top) <= (2.0 ** -9 + 2.0 ** -16) * np.abs(top)).all()
    assert (np.abs(lse - (15 * 2.0 ** 23 + np.log(60))) <= 2.0 ** -20 * 15 * 2.0 ** 23).all()


def check_long(q, lat, rope, o, lse, what):
    """test_gpu_fp4's bound for long sums and small weights. Per output element, with its A, B and C:
    * scores as there, E; a weight is off by 2^-11 of itself, or, below 2^-21 of the largest weight, by 2^-32 of the
      largest, which is at most the weights' sum: 2^-32 C;
    * O's N / 16 accumulations are off by 2^-22 of the sum of magnitudes each, the N additions of the weights' sum by
      2^-24 of it each, spread over six partial sums: N (2^-26 + 2^-26) A;
    * 2^-8 of o, the bf16 result. lse: E, the N 2^-26 of the sum, and 2^-20 (1 + |lse|)."""
    n = lat.shape[0]
    want, wlse, A, B = F.attend(T.bf16_decode(q), lat, rope, T.SM)
    E = 2.0 ** -16 * B
    bound = ((2 * E[:, None] + 2.0 ** -11 + 2.0 ** -16 + n * 2.0 ** -25) * A + 2.0 ** -32 * np.abs(lat).sum(0) +
             2.0 ** -8 * np.abs(want) + 1e-30)
    off = np.abs(o - want)
    assert (off <= bound).all(), f"{what}: {(off / bound).max()} of the bound, {np.linalg.norm(off) / np.linalg.norm(want)} of the norm"
    assert (np.abs(lse - wlse) <= E + n * 2.0 ** -26 + 2.0 ** -20 * (1 + np.abs(wlse))).all(), what
    return off, want


def behind_a_sink(rng, n, nats, jitter):
    """n rows of which the first is a sink: its score is `nats` above the others' (which differ by up to jitter), and it
    has no value in half of the latents. The others' latents are positive, so that their errors add up."""
    kv = np.zeros((n, 576))
    kv[:, :512] = rng.uniform(0.25, 1, (n, 512))
    kv[0, :256] = 0
    kv[1:, 513] = rng.uniform(-jitter, jitter, n - 1) / T.SM
    kv[0, 512] = nats / T.SM
    q = np.zeros((20, 576))
    q[:, 512:514] = 1
    return F.pack(T.bf16_bits(kv), 1.0), T.bf16_bits(q)


@pytest.mark.parametrize("nats", [10.0, 16.0, 18.0, 21.0])
@pytest.mark.parametrize("jitter", [0.0, 1.0])
def test_rows_behind_a_sink_keep_their_weight(nats, jitter):
    """Each of the others' weights is 2^-14 to 2^-30 of the sink's, which is seen first and sets the reference; half of
    the outputs are theirs alone. Through the row table and through the window, whole and split."""
    hs = T._gpu()
    rng = np.random.default_rng(int(nats))
    rec, q = behind_a_sink(rng, 4096, nats, jitter)
    lat, rope = F.unpack(rec, 1.0)
    rows = np.arange(4096, dtype=np.int32)[None]
    for splits in (1, 3):
        o, lse, err = T.sparse(hs, q[None], T.d(rec), T.d(rows), 1.0, splits)
        assert err == 0
        off, want = check_long(q, lat, rope, o[0], lse[0], f"row table, {splits} splits")
        if nats <= 18:
            assert (off[:, :256] <= 2.0 ** -5 * want[:, :256]).all()
    n = 32768
    rec, q = behind_a_sink(rng, n, nats, jitter)
    table, total = T.pages_for(rng, np.array([n], np.int32), 64, n // 64)
    pool = np.zeros((total, 416), np.uint8)
    pool[(table[0].astype(np.int64)[:, None] * 64 + np.arange(64)).reshape(-1)] = rec
    lat, rope = F.unpack(rec, 1.0)
    o, lse, err = T.window(hs, q[None, None], T.d(pool), 64, np.array([n], np.int32), table, n - 1, 1, 1.0, 1)
    assert err == 0
    check_long(q, lat, rope, o[0, 0], lse[0, 0], "window")


def test_a_window_over_a_whole_context_behind_a_sink():
    """131,072 rows of 2^-26 of the sink's weight each: together 2^-9 of the sum, and half of the outputs."""
    hs = T._gpu()
    rng = np.random.default_rng(1)
    n = 1 << 17
    rec, q = behind_a_sink(rng, n, 18.0, 0.0)
    table = np.arange(n // 64, dtype=np.int32)[None]
    o, lse, err = T.window(hs, q[None, None], T.d(rec), 64, np.array([n], np.int32), table, 2 ** 31 - 1, 1, 1.0, 1)
    assert err == 0
    lat, rope = F.unpack(rec, 1.0)
    off, want = check_long(q, lat, rope, o[0, 0], lse[0, 0], "whole context")
    assert (off[:, :256] <= 2.0 ** -5 * want[:, :256]).all()  # 2^-32 of 2^-25.97, 2^-8 twice, 2^-11: 0.024


@pytest.mark.parametrize("k", [-60, -30, -17, 17, 60, 100])
@pytest.mark.parametrize("splits", [1, 2])
def test_queries_of_any_size(k, splits):
    """A query times 2^k with a scale over 2^k has the same scores: the same bits, as nothing but exponents differ."""
    hs = T._gpu()
    q, pool, rows = T.case(13, 3, 40, 300, 500, g=0.5)
    want = T.sparse(hs, q, T.d(pool), T.d(rows), 0.5, splits)
    q2 = T.bf16_bits(T.bf16_decode(q) * 2.0 ** k)
    got = T.sparse(hs, q2, T.d(pool), T.d(rows), 0.5, splits, T.SM * 2.0 ** -k)
    for r in range(3):
        T.check(q[r], pool[rows[r][rows[r] >= 0]], 0.5, want[0][r], want[1][r], f"request {r}")
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1]) and got[2] == want[2] == 0


def test_queries_whose_values_differ_in_size():
    """Heads of 2^-20 beside heads of 2^40, latents from 2^-28 of a head's largest up to it, latents that are all zero,
    RoPE values 2^30 below and above the latents': the scores to test_gpu_fp4's E."""
    hs = T._gpu()
    rng = np.random.default_rng(17)
    _, pool, rows = T.case(19, 2, 1, 200, 300)
    q = rng.standard_normal((2, 40, 576))
    q[:, :, :512] *= 2.0 ** rng.integers(-28, 1, (2, 40, 512))
    q[:, 10:20, 512:] *= 2.0 ** -30
    q[:, 20:30, 512:] *= 2.0 ** 30
    q[:, 30:35, :512] = 0
    q *= 2.0 ** rng.integers(-20, 40, (2, 40, 1))
    q = T.bf16_bits(q)
    for sm in (T.SM, T.SM * 2.0 ** 20, T.SM * 2.0 ** -40):
        o, lse, err = T.sparse(hs, q, T.d(pool), T.d(rows), 1.0, 1, sm)
        assert err == 0
        for r in range(2):
            lat, rope = F.unpack(pool[rows[r][rows[r] >= 0]], 1.0)
            want, wlse, A, B = F.attend(T.bf16_decode(q[r]), lat, rope, sm)
            E = 2.0 ** -16 * B
            assert (np.abs(lse[r] - wlse) <= E + 2.0 ** -20 * (1 + np.abs(wlse))).all()
            sure = E < 2.0 ** -6  # where the scores decide anything
            bound = (2 * E[:, None] + 2.0 ** -10) * A + 2.0 ** -32 * np.abs(lat).sum(0) + 2.0 ** -8 * np.abs(want) + 1e-30
            assert (np.abs(o[r] - want) <= bound)[sure].all()
            assert (np.abs(o[r]) <= np.abs(lat).max(0) * (1 + 2.0 ** -7)).all()


@pytest.mark.parametrize("k", [0, 60, 100])
def test_a_scale_of_zero_weighs_rows_alike(k):
    """Whatever the query's size: o is the rows' mean, off by the weights' 2^-11, sums and the bf16 result; lse = log n."""
    hs = T._gpu()
    q, pool, rows = T.case(23, 2, 30, 300, 400, masked=0.0)
    q = T.bf16_bits(T.bf16_decode(q) * 2.0 ** k)
    for splits in (1, 2):
        o, lse, err = T.sparse(hs, q, T.d(pool), T.d(rows), 1.0, splits, 0.0)
        assert err == 0
        for r in range(2):
            lat, _ = F.unpack(pool[rows[r]], 1.0)
            mean, A = lat.mean(0), np.abs(lat).mean(0)
            assert (np.abs(o[r] - mean) <= (2.0 ** -11 + 2.0 ** -16) * A + 2.0 ** -8 * np.abs(mean) + 1e-30).all()
            assert (np.abs(lse[r] - np.log(300)) <= 2.0 ** -20 * 7).all()


def test_nan_in_one_warpgroups_blocks_reaches_the_sum():
    """A row whose score is NaN, alone in its block of 64 and so in one of three partial sums."""
    hs = T._gpu()
    q, pool, rows = T.case(29, 1, 20, 192, 300, masked=0.0)
    pool[7, 256:288] = 0x7F
    rows[rows == 7] = 8
    for block in range(3):
        named = rows.copy()
        named[0, 64 * block:64 * block + 64] = -1
        named[0, 64 * block + 5] = 7
        o, lse, err = T.sparse(hs, q, T.d(pool), T.d(named), 1.0, 1)
        assert err == 0 and np.isnan(o).all() and np.isnan(lse).all()


@pytest.mark.parametrize("splits", [1, 3])
def test_the_most_requests_of_a_call(splits):
    """2^20 requests of one head and up to two rows each (every third has one, every third none): o is the row where
    there is one, to the bf16 rounding, between the rows where there are two."""
    hs = T._gpu()
    R = hs.HS_MAX_FP4_MLA_REQUESTS
    rng = np.random.default_rng(37)
    rec = F.pack(T.tokens(rng, 500), 1.0)
    lat = torch.from_numpy(F.unpack(rec, 1.0)[0]).cuda().float()
    rows = torch.randint(0, 500, (R, 2), dtype=torch.int32, device="cuda")
    rows[0::3], rows[1::3, 1] = -1, -1
    q = torch.randn(R, 1, 576, device="cuda").to(torch.bfloat16)
    wsb = hs.hs_fp4_mla_workspace_bytes(R, 1, 1, splits)
    ws = torch.empty(max(16, wsb), dtype=torch.uint8, device="cuda")
    o, lse, err = torch.empty(R, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(R, 1, device="cuda"), T.flags()
    hs.hs_fp4_sparse_mla_decode(R, 1, 2, splits, q, T.d(rec), 500, rows, T.SM, 1.0, o, lse, ws, wsb, err)
    assert int(err.item()) == 0
    assert not o[0::3].any() and torch.isneginf(lse[0::3]).all()
    one = lat[rows[1::3, 0].long()]
    assert ((o[1::3].float() - one).abs() <= 2.0 ** -9 * one.abs()).all()
    a, b = lat[rows[2::3, 0].long()], lat[rows[2::3, 1].long()]
    slack = 2.0 ** -8 * torch.maximum(a.abs(), b.abs())
    got = o[2::3].float()
    assert ((got >= torch.minimum(a, b) - slack) & (got <= torch.maximum(a, b) + slack)).all()
    assert torch.isfinite(lse[1::3]).all() and torch.isfinite(lse[2::3]).all()


def test_the_most_entries_of_a_page_call():
    """2^20 entries, most of them padding: requests that grow stand far apart, a request is named twice, and a free
    names the same requests again and again."""
    hs = T._gpu()
    import test_gpu_pages as G
    n = hs.HS_MAX_PAGE_ENTRIES
    s = G.Pair(hs, 11, 40, 5, 120, 4)
    rng = np.random.default_rng(4)
    at = np.sort(rng.choice(n, 12, replace=False))
    at[-1] = n - 1
    r, new = np.full(n, -1, np.int32), np.zeros(n, np.int32)
    r[at], new[at] = [3, 4, 5, 6, 7, 8, 9, 10, 11, 9, 39, 12], [20, 7, 1, 0, 8, 20, 20, 20, 16, 4, 20, 3]
    got = torch.zeros(n, dtype=torch.int32, device="cuda")
    hs.hs_pages_extend(s.pool, n, G.d(r), G.d(np.zeros(n)), G.d(new), got)
    want, flags = s.orc.extend(r[at].tolist(), [0] * 12, new[at].tolist())
    assert got.cpu().numpy()[at].tolist() == want and int(got.abs().sum()) == np.abs(want).sum()
    s.same(flags)
    r = np.full(n, -1, np.int32)
    r[::7] = rng.choice([3, 5, 39, 2], r[::7].size)
    hs.hs_pages_free(s.pool, n, G.d(r))
    s.same(s.orc.release([3, 5, 39, 2]))
