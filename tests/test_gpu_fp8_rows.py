"""GPU parity of the fp8 rows against the oracle in 64 bits.

Codes and scales are equal, byte for byte: the kernel decides as exact arithmetic does for values that are not within
2^-44 of a border between two codes, and of these tests' (under 2^23) values some 2^23 x 2^-40 are expected to be.
RoPE values that are rotated: within half a step of bf16 (2^-8 of the value) of the exact ones, and 2^-22 of it for
the 32-bit sum before that rounding; below 2^-126 bf16's steps are 2^-133 whatever the value's size, half a step 2^-134,
and 32 bits add up to 3 x 2^-150 (a sum's and two products' half steps): 2^-133 in all covers values there.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import chunk as C  # noqa: E402
from oracle.sparse_mla import bf16_decode  # noqa: E402

pytestmark = pytest.mark.gpu


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


def flags():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def tokens(rng, n, scale=1.0):
    x = rng.standard_normal((n, 576)) * scale
    x[:, :512:37] *= 6
    x[:, 5:512:11] *= 0.05
    return bits(x)


def rope_table(n):
    ang = np.arange(n)[:, None] * 10000.0 ** (-np.arange(0, 64, 2) / 64.0)
    return np.concatenate((np.cos(ang), np.sin(ang)), 1).astype(np.float32)


def same_rows(got, want):
    """got rows [n, 656] against the oracle's (codes and scales, RoPE values)."""
    rec, rope = want
    assert np.array_equal(got[:, :512], rec[:, :512])
    a, b = got[:, 512:528].copy().view(np.float32), rec[:, 512:].copy().view(np.float32)
    assert np.array_equal(a, b, equal_nan=True)
    r = bf16_decode(got[:, 528:].copy().view("<u2"))
    fine = np.isfinite(rope)
    assert np.array_equal(np.isnan(r), np.isnan(rope)) and np.array_equal(r[~fine & ~np.isnan(rope)], rope[~fine & ~np.isnan(rope)])
    assert (np.abs(r - rope)[fine] <= (2.0 ** -8 + 2.0 ** -22) * np.abs(rope[fine]) + 2.0 ** -133).all()


@pytest.mark.parametrize("n,stride,norm,rotate,scale", [(1, 576, True, True, 1.0), (3, 640, False, False, 1.0), (33, 576, True, False, 100.0), (257, 1088, False, True, 2.0 ** -60),
                                                        (1025, 584, True, True, 1e-3), (64, 576, True, True, 2.0 ** 90), (64, 576, True, True, 2.0 ** -90)])
def test_rows_written_and_read_back(n, stride, norm, rotate, scale):
    hs = _gpu()
    rng = np.random.default_rng(n + stride)
    kv = np.full((n, stride), 0x7FC0, np.uint16)  # past 576: not read
    kv[:, :576] = tokens(rng, n, scale)
    total = 2 * n + 5
    rows = rng.permutation(total)[:n].astype(np.int32)
    pos = rng.integers(0, 5000, n).astype(np.int32)
    want_flags = 0
    if n > 5:
        rows[1], rows[2] = -1, total
        want_flags |= hs.HS_FLAG_DEVROW
        if rotate:
            pos[3], pos[4] = -1, 5000
            want_flags |= hs.HS_FLAG_SEQLEN
    if n > 40 and scale == 1e-3:
        kv[5, 17], kv[6, 130], kv[7, 500] = 0x7FC0, 0x7F80, 0xFF80
        kv[8, :512] = 0
        kv[9, 128:256] = 0x8000
        kv[10, 512:520] = [0x7F80, 0, 0x7FC0, 0, 0, 0x8000, 1, 2]
    w = bits(1 + 0.3 * rng.standard_normal(512)) if norm else None
    table = rope_table(5000) if rotate else None
    pool0 = rng.integers(0, 256, (total, 656)).astype(np.uint8)
    pool, err = d(pool0), flags()
    hs.hs_fp8_pack_rows(n, d(kv), stride, d(rows), d(w) if norm else None, 1e-6, d(pos) if rotate else None, d(table) if rotate else None, 5000, pool, total, err)
    ok = (rows >= 0) & (rows < total)
    if rotate:
        ok &= (pos >= 0) & (pos < 5000)
    got = pool.cpu().numpy()
    same_rows(got[rows[ok]], C.pack(kv[ok, :576], w, 1e-6, pos[ok], table))
    rest = np.ones(total, bool)
    rest[rows[ok]] = False
    assert np.array_equal(got[rest], pool0[rest]) and int(err.item()) == want_flags
    # back: rows of any scale, some twice, some absent
    rec = got.copy()
    rec[rest, 512:528] = rng.standard_normal((int(rest.sum()), 4)).astype(np.float32).view(np.uint8)
    rec[rest, 528:] = tokens(rng, int(rest.sum()))[:, :64].view(np.uint8)
    back = rng.integers(-1, total, 3 * n + 1).astype(np.int32)
    back[0] = total + 7
    out, err = torch.full((back.size, stride), 123, dtype=torch.int16, device="cuda"), flags()
    hs.hs_fp8_unpack_rows(back.size, d(rec), total, d(back), out, stride, err)
    live = (back >= 0) & (back < total)
    lat, rope = C.unpack(rec[np.where(live, back, 0)])
    with np.errstate(over="ignore"):
        want = np.where(live[:, None], bf16_decode(bits(np.concatenate((lat, rope), 1))), 0)
    o = out.cpu().numpy().view(np.uint16)
    val = bf16_decode(o[:, :576])
    exact = np.where(live[:, None], np.concatenate((lat, rope), 1), 0)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(val), np.isnan(want)) and (np.abs(val - exact)[fine] <= (2.0 ** -8 + 2.0 ** -23) * np.abs(exact[fine]) + 2.0 ** -134).all()
    written = live & ~rest[np.where(live, back, 0)]
    assert np.array_equal(val[written], exact[written], equal_nan=True)  # powers of two: exact
    assert (o[:, 576:] == 123).all() and int(err.item()) == hs.HS_FLAG_DEVROW


def test_values_around_every_border():
    """Without a norm: every bf16 value of nine binades beside a block's largest, which sets the scale: halfway points of
    e4m3, its subnormal range, values that round to zero."""
    hs = _gpu()
    v = (np.arange(0x3B00, 0x4400, dtype=np.uint32) << 16).view(np.float32)  # 2^-9 .. 2^9
    n = 64
    kv = np.zeros((n, 576), np.float32)
    flat = np.resize(np.concatenate((v, -v)), (n, 4, 127))
    lat = np.zeros((n, 4, 128), np.float32)
    lat[..., 1:] = flat
    lat[..., 0] = np.resize([512.0, 448.0, 450.0, 3.0, 900.0], (n, 4))
    kv[:, :512] = lat.reshape(n, 512)
    kb = bits(kv)
    pool = torch.zeros(n, 656, dtype=torch.uint8, device="cuda")
    hs.hs_fp8_pack_rows(n, d(kb), 576, torch.arange(n, dtype=torch.int32, device="cuda"), None, 0.0, None, None, 0, pool, n, flags())
    same_rows(pool.cpu().numpy(), C.pack(kb))


def test_a_norm_decides_as_exact_arithmetic_at_borders():
    """Tokens whose norm is a power of two exactly (512 values of the same magnitude, no eps), times weights: values on
    halfway points go to the even code, and weights one bf16 step around them to their sides."""
    hs = _gpu()
    n = 128
    mag = bits(2.0 ** (np.arange(n) % 40 - 20))
    kv = np.zeros((n, 576), np.uint16)
    kv[:, :512] = mag[:, None]
    kv[1::2, :512:3] |= 0x8000
    w = bits(np.resize(np.concatenate([m * 2.0 ** e * np.array([1 - 2.0 ** -7, 1.0, 1 + 2.0 ** -7]) for e in (-6, -2, 0, 3, 8) for m in (17 / 16, 19 / 16, 31 / 16, 1.75)]), 512))
    pool = torch.zeros(n, 656, dtype=torch.uint8, device="cuda")
    hs.hs_fp8_pack_rows(n, d(kv), 576, torch.arange(n, dtype=torch.int32, device="cuda"), d(w), 0.0, None, None, 0, pool, n, flags())
    same_rows(pool.cpu().numpy(), C.pack(kv, w, 0.0))


def test_rows_past_four_gigabytes():
    hs = _gpu()
    total = 7_000_000  # 4.6 GB
    pool = torch.empty(total, 656, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(9)
    kv = tokens(rng, 40)
    rows = np.concatenate((np.arange(20), np.arange(total - 20, total))).astype(np.int32)[rng.permutation(40)]
    hs.hs_fp8_pack_rows(40, d(kv), 576, d(rows), None, 0.0, None, None, 0, pool, total, flags())
    got = pool[d(rows).long()].cpu().numpy()
    same_rows(got, C.pack(kv))
    out = torch.zeros(40, 576, dtype=torch.int16, device="cuda")
    hs.hs_fp8_unpack_rows(40, pool, total, d(rows), out, 576, flags())
    assert np.array_equal(bf16_decode(out.cpu().numpy().view(np.uint16)), np.concatenate(C.unpack(got), 1))


def test_a_norm_of_a_million_values_has_the_oracle_s_codes():
    hs = _gpu()
    rng = np.random.default_rng(10)
    n = 2048
    kv, w = tokens(rng, n), bits(1 + 0.3 * rng.standard_normal(512))
    pool = torch.zeros(n, 656, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    args = [d(kv), 576, torch.arange(n, dtype=torch.int32, device="cuda"), d(w), 1e-6, None, None, 0, pool, n, flags()]
    torch.cuda.synchronize()
    hs.hs_fp8_pack_rows(n, *args, stream=side)
    side.synchronize()
    same_rows(pool.cpu().numpy(), C.pack(kv, w, 1e-6))
