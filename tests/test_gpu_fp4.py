"""GPU parity of the 4-bit rows and the attention over them against the oracle in 64 bits.

Rows: bytes are equal (the kernel's 32-bit arithmetic gives the exact quotients' roundings).

Attention, per output element, with A_i = sum_j p_j |latent_ji| and B = max_j sm sum_d |q_d k_jd|:
* scores: products of 16-bit values are exact in the accumulator, 36 accumulations of up to 16
  products each round (or truncate) by at most 2^-22 of sum |q_d k_d|, (36 + 16) 2^-22 < 2^-16:
  E = 2^-16 B, and q and RoPE values under 2^-14 (none in these inputs but zeros) would add theirs;
* weights: exp of a score off by E is off by E relative, 2 E after normalising; a weight rounded
  to fp16 is off by 2^-11: together |d o_i| <= (2 E + 2^-11 + 2^-16) A_i, 2^-16 for the sums;
* small weights: below 2^-14 of the reference maximum's weight fp16 is subnormal, in steps of 2^-24,
  so a weight is off by up to 2^-25 whatever its size. The reference maximum is a score that the
  query saw, so the weights' sum is at least 1: |d o_i| <= 2^-25 C_i more, C_i = sum_j |latent_ji|
  (a dim that only rows of small weight have a value in shows it, as A_i is tiny there);
* the bf16 result: 2^-8 |o_i|;
* lse: |d| <= E + 2^-20 (1 + |lse|), the 32-bit logarithm and sum.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import fp4_mla as F  # noqa: E402
from oracle.sparse_mla import bf16_decode  # noqa: E402

pytestmark = pytest.mark.gpu
SM = 0.0722


def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hierarchical_sparse_attention_gb300 as hs
    return hs


def bf16_bits(x):
    return (torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).view(torch.int16).numpy()
            .view(np.uint16))


def d(x):
    x = np.ascontiguousarray(x)
    if x.dtype == np.uint16:
        x = x.view(np.int16)
    return torch.from_numpy(x).cuda()


def tokens(rng, n):
    x = rng.standard_normal((n, 576))
    x[:, :512:37] *= 6
    x[:, 5:512:11] *= 0.05
    return bf16_bits(x)


def flags():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ rows


@pytest.mark.parametrize("n,stride,g", [(1, 576, 1.0), (3, 640, 0.25), (33, 576, 2.0 ** -20), (257, 1088, 8.0), (2048, 584, 1.0)])
def test_rows_written_and_read_back(n, stride, g):
    hs = _gpu()
    rng = np.random.default_rng(n)
    kv = np.zeros((n, stride), np.uint16)
    kv[:, :576] = bf16_bits(bf16_decode(tokens(rng, n)) * g)
    kv[:, 576:] = 0x7FC0  # not read
    total = 2 * n + 5
    rows = rng.permutation(total)[:n].astype(np.int32)
    if n > 3:
        rows[1] = -1
        rows[2] = total  # past the pool
        special = kv[0].view(np.uint16)
        special[:16] = 0
        special[16:32] = bf16_bits(np.full(16, 2.0 ** -30 * g))  # scale rounds to zero
        special[35], special[52], special[70] = 0x7FC0, 0x7F80, 0xFF80  # NaN, +inf, -inf
        special[80:96] = bf16_bits(np.full(16, 2.0 ** 60 * g))  # saturates
        special[96:112] = bf16_bits(np.array([6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25] * 2) * g)  # halfway, to the even code
        special[104:112] |= 0x8000
        special[112:128] = bf16_bits(np.full(16, 6.375 * 2.0 ** -10 * g))  # a subnormal scale's halfway point and beyond
        special[128:144] = 0x8000  # -0
        special[512:516] = [0x7FC0, 0x7F80, 0x0001, 0x8000]  # RoPE values are copied as they are
    pool0 = rng.integers(0, 256, (total, 416)).astype(np.uint8)
    pool, err = d(pool0), flags()
    hs.hs_fp4_pack_rows(n, d(kv), stride, d(rows), g, pool, total, err)
    want = pool0.copy()
    ok = (rows >= 0) & (rows < total)
    want[rows[ok]] = F.pack(kv[ok, :576], g)
    assert np.array_equal(pool.cpu().numpy(), want)
    assert int(err.item()) == (hs.HS_FLAG_DEVROW if (rows >= total).any() else 0)
    # back: every row, some twice, some absent
    want = np.where(np.arange(total)[:, None] % 3 == 0, want, F.pack(tokens(rng, total), g))
    back = rng.integers(-1, total, 3 * n + 1).astype(np.int32)
    back[0] = total + 7
    out = torch.full((back.size, stride), 123, dtype=torch.int16, device="cuda")
    err = flags()
    pool = d(np.where((want[:, 256:288] & 0x7F == 0x7F).any(1)[:, None], F.pack(tokens(rng, total), g), want))
    hs.hs_fp4_unpack_rows(back.size, pool, total, d(back), g, out, stride, err)
    live = (back >= 0) & (back < total)
    lat, rope = F.unpack(pool.cpu().numpy()[np.where(live, back, 0)], g)
    val = np.where(live[:, None], np.concatenate((lat, rope), 1), 0)
    got = out.cpu().numpy().view(np.uint16)
    got_val = bf16_decode(got[:, :576])
    assert np.array_equal(got_val, val, equal_nan=True)
    assert (got[:, 576:] == 123).all() and int(err.item()) == hs.HS_FLAG_DEVROW


def test_every_bf16_magnitude_against_every_scale_rounds_as_the_oracle():
    """Each block holds a maximum and fifteen other values over eight binades: all 128 mantissas of the
    maximum, so every scale mantissa, and values on both sides of every halfway point."""
    hs = _gpu()
    top = (np.arange(128, dtype=np.uint32) << 16 | 0x40000000).view(np.float32)  # 2 .. 4
    kv = np.zeros((512, 576), np.uint16)
    v = np.empty((512, 32, 16), np.float32)
    v[..., 0] = np.resize(top, (512, 32))
    frac = (np.arange(512 * 32 * 15) % 1021).reshape(512, 32, 15) / 1020.0
    v[..., 1:] = v[..., :1] * frac
    kv[:, :512] = bf16_bits(v.reshape(512, 512))
    pool = torch.zeros(512, 416, dtype=torch.uint8, device="cuda")
    hs.hs_fp4_pack_rows(512, d(kv), 576, torch.arange(512, dtype=torch.int32, device="cuda"), 1.0, pool, 512, flags())
    assert np.array_equal(pool.cpu().numpy(), F.pack(kv, 1.0))


def test_rows_past_four_gigabytes():
    hs = _gpu()
    total = 11_000_000  # 4.6 GB
    pool = torch.empty(total, 416, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(9)
    kv = tokens(rng, 40)
    rows = np.concatenate((np.arange(20), np.arange(total - 20, total))).astype(np.int32)[rng.permutation(40)]
    err = flags()
    hs.hs_fp4_pack_rows(40, d(kv), 576, d(rows), 1.0, pool, total, err)
    assert np.array_equal(pool[d(rows).long()].cpu().numpy(), F.pack(kv, 1.0))
    out = torch.zeros(40, 576, dtype=torch.int16, device="cuda")
    hs.hs_fp4_unpack_rows(40, pool, total, d(rows), 1.0, out, 576, err)
    rec = F.pack(kv, 1.0)
    assert np.array_equal(bf16_decode(out.cpu().numpy().view(np.uint16)), np.concatenate(F.unpack(rec, 1.0), 1))
    q = bf16_bits(rng.standard_normal((1, 16, 576)))
    o, lse, e = sparse(hs, q, pool, d(rows[None]), 1.0, 2)
    check(q[0], rec, 1.0, o[0], lse[0], "past 4 GB")
    assert e == 0 and int(err.item()) == 0


# ------------------------------------------------------------------ attention


def buffers(hs, R, H, Q, splits):
    wsb = hs.hs_fp4_mla_workspace_bytes(R, H, Q, splits)
    return (torch.full((R, Q, H, 512), float("nan"), dtype=torch.bfloat16, device="cuda"),
            torch.full((R, Q, H), float("nan"), dtype=torch.float32, device="cuda"),
            torch.full((max(wsb, 16),), 255, dtype=torch.uint8, device="cuda"), wsb)


def sparse(hs, q, pool, rows, g, splits, sm=SM):
    R, H, _ = q.shape
    o, lse, ws, wsb = buffers(hs, R, H, 1, splits)
    err = flags()
    hs.hs_fp4_sparse_mla_decode(R, H, rows.shape[1], splits, d(q), pool, pool.shape[0], rows, sm, g, o, lse, ws, wsb, err)
    torch.cuda.synchronize()
    return o[:, 0].float().cpu().numpy(), lse[:, 0].cpu().numpy(), int(err.item())


def window(hs, q, pool, page, lens, table, W, sinks, g, splits, sm=SM):
    R, Q, H, _ = q.shape
    o, lse, ws, wsb = buffers(hs, R, H, Q, splits)
    err = flags()
    hs.hs_fp4_window_mla_decode(R, H, Q, W, sinks, splits, d(q), pool, pool.shape[0], page, table.shape[1], d(lens),
                                d(table), sm, g, o, lse, ws, wsb, err)
    torch.cuda.synchronize()
    return o.float().cpu().numpy(), lse.cpu().numpy(), int(err.item())


def check(q_bits, rec, g, o, lse, what, sm=SM):
    """q_bits [M, 576] over the rows rec [n, 416]."""
    lat, rope = F.unpack(rec, g)
    want, wlse, A, B = F.attend(bf16_decode(q_bits), lat, rope, sm)
    if rec.shape[0] == 0:
        assert (o == 0).all() and np.isneginf(lse).all(), what
        return
    E = 2.0 ** -16 * B
    bound = (2 * E[:, None] + 2.0 ** -11 + 2.0 ** -16) * A + 2.0 ** -25 * np.abs(lat).sum(0) + 2.0 ** -8 * np.abs(want) + 1e-30
    off = np.abs(o - want)
    assert (off <= bound).all(), f"{what}: o off by {off.max()}, {(off / bound).max()} of the bound"
    off = np.abs(lse - wlse)
    assert (off <= E + 2.0 ** -20 * (1 + np.abs(wlse))).all(), f"{what}: lse off by {off.max()}"


def case(seed, R, H, K, total, masked=0.1, g=1.0, Q=None):
    rng = np.random.default_rng(seed)
    pool = F.pack(bf16_bits(bf16_decode(tokens(rng, total)) * g), g)
    rows = rng.integers(0, total, (R, K)).astype(np.int32)
    rows[rng.random((R, K)) < masked] = -1
    q = bf16_bits(rng.standard_normal((R, H, 576) if Q is None else (R, Q, H, 576)))
    return q, pool, rows


@pytest.mark.parametrize("R,H,K,splits,g", [(1, 1, 1, 1, 1.0), (2, 16, 64, 1, 0.25), (3, 128, 65, 1, 1.0), (2, 128, 256, 1, 1.0),
                                            (2, 128, 2048, 2, 1.0), (2, 64, 100, 3, 8.0), (1, 7, 333, 4, 2.0 ** -20),
                                            (2, 127, 600, 16, 1.0), (2, 128, 5, 16, 1.0), (2, 48, 4096, 1, 1.0),
                                            (3, 17, 4095, 2, 1.0), (90, 128, 130, 2, 1.0), (200, 8, 70, 1, 1.0),
                                            (40, 33, 200, 4, 1.0)])
def test_sparse_matches_the_oracle(R, H, K, splits, g):
    hs = _gpu()
    q, pool, rows = case(R * 7 + K, R, H, K, 1500, g=g)
    o, lse, err = sparse(hs, q, d(pool), d(rows), g, splits, SM / max(g, 1e-3))
    assert err == 0
    for r in range(R):
        check(q[r], pool[rows[r][rows[r] >= 0]], g, o[r], lse[r], f"request {r}", SM / max(g, 1e-3))


@pytest.mark.parametrize("splits", [1, 2, 5])
def test_sparse_rows_left_out(splits):
    """Requests with no row, rows past the pool, one row many times, and NaN and infinities in rows
    that are not named."""
    hs = _gpu()
    q, pool, rows = case(5, 5, 40, 200, 500, masked=0.5)
    pool[7, 256:288] = 0x7F  # NaN latents
    pool[8, 288:] = np.tile(np.array([0x80, 0x7F], np.uint8), 64)  # inf RoPE
    rows[(rows == 7) | (rows == 8)] = 9
    rows[0, :17] = 505
    rows[0, 17:20] = np.iinfo(np.int32).max
    rows[1] = -1
    rows[2] = 11
    rows[3, 1:] = np.iinfo(np.int32).min
    rows[3, 0] = 499
    o, lse, err = sparse(hs, q, d(pool), d(rows), 1.0, splits)
    assert err == 0
    for r in range(5):
        check(q[r], pool[rows[r][(rows[r] >= 0) & (rows[r] < 500)]], 1.0, o[r], lse[r], f"request {r}")
    rows[4, 100] = 7  # named: the request's outputs are NaN, the others' are not
    o2, lse2, _ = sparse(hs, q, d(pool), d(rows), 1.0, splits)
    assert np.isnan(o2[4]).all() and np.isnan(lse2[4]).all()
    assert np.array_equal(o2[:4], o[:4]) and np.array_equal(lse2[:4], lse[:4])


@pytest.mark.parametrize("order", ["rising", "falling", "late spike"])
@pytest.mark.parametrize("splits", [1, 2])
def test_sparse_running_maximum(order, splits):
    """Scores that rise by hundreds over the rows, fall, or jump once near the end."""
    hs = _gpu()
    rng = np.random.default_rng(4)
    kv = np.zeros((1000, 576))
    kv[:, :512] = rng.standard_normal((1000, 512))
    slope = {"rising": np.arange(1000), "falling": np.arange(1000)[::-1], "late spike": np.where(np.arange(1000) == 901, 800, 0)}
    kv[:, 512] = slope[order] // 4  # bf16 holds these
    pool = F.pack(bf16_bits(kv), 1.0)
    q = bf16_bits(rng.standard_normal((1, 32, 576)))
    q[:, :, 512] = bf16_bits(np.full((1, 32), 16.0))
    o, lse, err = sparse(hs, q, d(pool), torch.arange(1000, dtype=torch.int32, device="cuda")[None].contiguous(), 1.0, splits)
    assert err == 0
    check(q[0], pool, 1.0, o[0], lse[0], order)


def pages_for(rng, lens, page, max_pages, spare=3):
    """A page table that holds every token, its pages in any order, and the pool's rows."""
    held = -(-np.maximum(lens, 0) // page)
    total = int(held.sum()) + spare
    perm = rng.permutation(total).astype(np.int32)
    table = np.full((len(lens), max_pages), -1, np.int32)
    at = 0
    for r, n in enumerate(held):
        table[r, :n] = perm[at:at + n]
        at += n
    return table, total * page


def check_window(q, pool, page, lens, table, W, sinks, g, o, lse, sm=SM):
    R, Q, H, _ = q.shape
    for r in range(R):
        for i in range(Q):
            t = F.window_tokens(int(lens[r]) - Q + i, W, sinks)
            pg = table[r, t // page].astype(np.int64)
            rows = (pg * page + t % page)[(pg >= 0) & (pg * page + t % page < pool.shape[0])]
            check(q[r, i], pool[rows], g, o[r, i], lse[r, i], f"request {r} query {i}", sm)


@pytest.mark.parametrize("H,Q,W,sinks,page,splits,lens", [
    (16, 1, 127, 3, 64, 1, (1000, 1, 64, 128, 0)),
    (128, 1, 100, 0, 16, 1, (300, 99, 100, 101)),
    (128, 1, 1, 0, 64, 1, (1, 65, 500)),
    (128, 3, 70, 4, 64, 2, (500, 2, 3, 75)),
    (16, 4, 64, 4, 48, 1, (500, 1, 2, 3, 4, 5, 66, 68, 72, 0)),
    (8, 8, 33, 1, 1, 3, (200, 8, 7, 40)),
    (3, 8, 1000, 64, 128, 16, (2000, 1500, 63, 65, 1064)),
    (128, 2, 3000, 8, 64, 4, (5000, 2999)),
    (37, 5, 200, 100, 7, 2, (1000, 100, 99, 300, 301)),
    (64, 1, 5000, 64, 64, 1, (6000, 4096)),
    (1, 1, 2 ** 31 - 1, 2 ** 31 - 1, 64, 2, (700, 1))])
def test_window_matches_the_oracle(H, Q, W, sinks, page, splits, lens):
    hs = _gpu()
    rng = np.random.default_rng(W % 1000 + H)
    lens = np.array(lens, np.int32)
    table, rows = pages_for(rng, lens, page, -(-int(lens.max()) // page) + 2)
    q, pool, _ = case(H + Q, len(lens), H, 1, rows, g=0.5, Q=Q)
    o, lse, err = window(hs, q, d(pool), page, lens, table, W, sinks, 0.5, splits)
    assert err == 0
    check_window(q, pool, page, lens, table, W, sinks, 0.5, o, lse)


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("H,Q", [(16, 4), (128, 2)])
def test_window_missing_pages_and_bad_lengths(H, Q, splits):
    hs = _gpu()
    rng = np.random.default_rng(8)
    page, W, sinks = 16, 90, 20
    lens = np.array([300, 300, 300, 300, 300], np.int32)
    table, rows = pages_for(rng, lens, page, 20)
    q, pool, _ = case(6, 5, H, 1, rows, Q=Q)
    lens2 = lens.copy()
    table[0, 3:12] = -1  # between the sinks and the window: nobody looks
    o, lse, err = window(hs, q, d(pool), page, lens, table, W, sinks, 1.0, splits)
    assert err == 0
    check_window(q, pool, page, lens, table, W, sinks, 1.0, o, lse)
    table[1, 1] = -1  # sink tokens 16 .. 19
    table[2, 17] = rows // page + 4  # past the pool
    table[2, 18] = np.iinfo(np.int32).max
    table[3, :] = -7  # nothing at all
    lens2[4] = 321  # longer than its table row
    o, lse, err = window(hs, q, d(pool), page, lens2, table, W, sinks, 1.0, splits)
    assert err == hs.HS_FLAG_DEVROW | hs.HS_FLAG_SEQLEN
    check_window(q[:4], pool, page, lens2[:4], table[:4], W, sinks, 1.0, o[:4], lse[:4])
    assert (o[4] == 0).all() and np.isneginf(lse[4]).all()
    lens2[4] = -1
    o, lse, err = window(hs, q, d(pool), page, lens2, table, W, sinks, 1.0, splits)
    assert err == hs.HS_FLAG_DEVROW | hs.HS_FLAG_SEQLEN
    assert (o[4] == 0).all() and np.isneginf(lse[4]).all()


@pytest.mark.parametrize("H,Q", [(16, 4), (128, 4)])
def test_window_nan_rows_that_some_queries_see(H, Q):
    """A verify step's later tokens, and the oldest token of the window, are seen by some queries of a
    request only: NaN and infinities in them reach those queries and no other."""
    hs = _gpu()
    rng = np.random.default_rng(2)
    lens = np.array([200], np.int32)
    table, rows = pages_for(rng, lens, 16, 13)
    q, pool, _ = case(1, 1, H, 1, rows, Q=Q)
    row = lambda t: int(table[0, t // 16]) * 16 + t % 16  # noqa: E731
    clean = window(hs, q, d(pool), 16, lens, table, 50, 2, 1.0, 2)
    bad = pool.copy()
    bad[row(199), 256:288] = 0x7F  # the last draft's latents
    bad[row(198), 288:] = np.tile(np.array([0x80, 0x7F], np.uint8), 64)  # the draft before it: inf RoPE
    bad[row(147), 256] = 0x7F  # token 147 is in the window of query 0 (token 196) only
    o, lse, err = window(hs, q, d(bad), 16, lens, table, 50, 2, 1.0, 2)
    assert err == 0
    assert np.isnan(lse[0, 0]).all() and np.isnan(o[0, 0]).all()
    assert np.array_equal(o[0, 1], clean[0][0, 1]) and np.array_equal(lse[0, 1], clean[1][0, 1])
    assert np.isnan(o[0, 3]).all() and np.isnan(lse[0, 3]).all()
    assert not np.isfinite(lse[0, 2]).all()


def test_calls_on_a_stream_and_from_a_replayed_graph():
    """Two captured calls that share a workspace, replayed with other inputs, give what eager calls on
    another stream give, bit for bit."""
    hs = _gpu()
    rng = np.random.default_rng(3)
    R, H, Q, K = 6, 32, 3, 500
    lens = np.array([700, 650, 3, 0, 512, 90], np.int32)
    table, rows = pages_for(rng, lens, 64, 12)
    q1, pool, tab = case(2, R, H, K, rows)
    q2 = case(4, R, H, 1, 10, Q=Q)[0]
    g_q1, g_q2, g_pool, g_tab, g_lens, g_table = d(q1), d(q2), d(pool), d(tab), d(lens), d(table)
    splits = 3
    wsb = max(hs.hs_fp4_mla_workspace_bytes(R, H, Q, splits), hs.hs_fp4_mla_workspace_bytes(R, H, 1, splits))

    def outputs():
        return [torch.full((R, H, 512), float("nan"), dtype=torch.bfloat16, device="cuda"), torch.zeros(R, H, device="cuda"),
                torch.full((R, Q, H, 512), float("nan"), dtype=torch.bfloat16, device="cuda"), torch.zeros(R, Q, H, device="cuda"),
                torch.full((wsb,), 255, dtype=torch.uint8, device="cuda"), flags()]

    def calls(o, s):
        hs.hs_fp4_sparse_mla_decode(R, H, K, splits, g_q1, g_pool, rows, g_tab, SM, 1.0, o[0], o[1], o[4], wsb, o[5], stream=s)
        hs.hs_fp4_window_mla_decode(R, H, Q, 200, 5, splits, g_q2, g_pool, rows, 64, 12, g_lens, g_table, SM, 1.0, o[2], o[3],
                                    o[4], wsb, o[5], stream=s)

    a, b = outputs(), outputs()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        calls(a, s)
    for k in range(3):
        g_q1.copy_(g_q1.flip(0))
        g_lens.copy_(g_lens.roll(1) if k == 2 else g_lens)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        other = torch.cuda.Stream()
        calls(b, other)
        torch.cuda.synchronize()
        for x, y in zip(a[:4], b[:4]):
            assert torch.equal(x, y)
    assert int(a[5].item()) == int(b[5].item())


def test_splits_and_workspaces():
    hs = _gpu()
    for R, H, Q, rows in ((1, 16, 1, 64), (32, 128, 1, 2048), (256, 128, 1, 2048), (1, 128, 1, 1 << 20), (64, 16, 8, 9000)):
        s = hs.hs_fp4_mla_splits(R, H, Q, rows)
        assert 1 <= s <= hs.HS_MAX_MLA_SPLITS
        assert (hs.hs_fp4_mla_workspace_bytes(R, H, Q, s) > 0) == (s > 1)
