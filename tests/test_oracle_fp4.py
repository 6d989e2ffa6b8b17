"""What pins the 4-bit oracle and the page oracle, and the host-side refusals of their calls (no GPU)."""
import ctypes
import math

import numpy as np
import pytest

from oracle import fp4_mla as F
from oracle import pages as P


def bits(x):
    """bf16 bit patterns of float32 values that bf16 holds exactly."""
    b = np.asarray(x, np.float32).view(np.uint32)
    assert not (b & 0xFFFF).any()
    return (b >> 16).astype(np.uint16)


def test_nearest_code_landmarks():
    x = np.array([0, 0.25, 0.2500001, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 5.1, 100.0])
    assert F.nearest_code(x, F.E2M1).tolist() == [0, 0, 1, 2, 2, 4, 4, 6, 6, 7, 7]
    assert F.E4M3[0] == 0 and F.E4M3[1] == 2.0 ** -9 and F.E4M3[126] == 448


@pytest.mark.parametrize("g", [2.0 ** -3, 1.0, 2.0 ** 7])
def test_pack_keeps_representable_values_and_is_within_half_a_step(g):
    rng = np.random.default_rng(3)
    # values that the format holds: code x scale, with a 6 in every block so that the scale comes out
    code = rng.integers(0, 16, (5, 32, 16))
    code[..., 3] = 7
    scale = rng.integers(8, 100, (5, 32))
    val = (F.E2M1[code & 7] * np.where(code & 8, -1, 1) * F.E4M3[scale][..., None] * g).reshape(5, 512)
    kv = np.concatenate((val, rng.integers(-8, 8, (5, 64))), 1)
    lat, rope = F.unpack(F.pack(bits(kv), g), g)
    assert np.array_equal(lat, val) and np.array_equal(rope, kv[:, 512:])
    # values of spread g, whose scales are normal e4m3 numbers: off by at most half the widest step
    # (6 - 4 = 2 scales) of their block
    kv = ((rng.standard_normal((5, 576)) * g).astype(np.float32).view(np.uint32) & 0xFFFF0000).view(np.float32)
    rec = F.pack(bits(kv), g)
    lat, _ = F.unpack(rec, g)
    s = np.repeat(F.e4m3_decode(rec[:, 256:288]), 16, 1) * g
    # the scale may be rounded down by 2^-4: the largest value then saturates at 6 scales of a needed 6 / (1 - 2^-4)
    assert (np.abs(lat - kv[:, :512]) <= s).all()


def test_pack_of_zeros_tiny_nan_and_infinite_blocks():
    kv = np.zeros((1, 576), np.uint16)
    kv[0, 16:32] = bits(2.0 ** -30)  # scale rounds to zero
    kv[0, 40] = 0x7FC0  # NaN
    kv[0, 50] = 0xFF80  # -inf
    kv[0, 64:80] = bits(2.0 ** 100)  # saturates
    rec = F.pack(kv, 1.0)
    lat, _ = F.unpack(rec, 1.0)
    assert (lat[0, :32] == 0).all() and np.isnan(lat[0, 32:64]).all() and (lat[0, 64:80] == 6 * 448).all()
    assert rec[0, 256 + 2] == 0x7F and (rec[0, 16:24] == 0).all()


def test_attention_closed_forms():
    rng = np.random.default_rng(0)
    lat, rope = rng.standard_normal((7, 512)), rng.standard_normal((7, 64))
    q = rng.standard_normal((3, 576))
    o, lse, _, _ = F.attend(q, lat[:1], rope[:1], 0.1)
    assert np.allclose(o, lat[0]) and np.allclose(lse, 0.1 * (q[:, :512] @ lat[0] + q[:, 512:] @ rope[0]))
    o, lse, _, _ = F.attend(np.zeros((1, 576)), lat, rope, 1.0)
    assert np.allclose(o[0], lat.mean(0)) and np.allclose(lse, math.log(7))
    parts = [F.attend(q, lat[a:b], rope[a:b], 0.1) for a, b in ((0, 3), (3, 7))]
    w = np.exp(np.stack([p[1] for p in parts]))
    whole = F.attend(q, lat, rope, 0.1)
    assert np.allclose((w[..., None] * np.stack([p[0] for p in parts])).sum(0) / w.sum(0)[:, None], whole[0])
    assert np.allclose(np.log(w.sum(0)), whole[1])


def test_window_tokens():
    assert F.window_tokens(-1, 4, 2).tolist() == []
    assert F.window_tokens(2, 4, 2).tolist() == [0, 1, 2]
    assert F.window_tokens(9, 4, 2).tolist() == [0, 1, 6, 7, 8, 9]
    assert F.window_tokens(9, 1, 0).tolist() == [9]
    assert F.window_tokens(3, 100, 100).tolist() == [0, 1, 2, 3]


def test_page_oracle_by_hand():
    pool = np.arange(8 * 4, dtype=np.uint8).reshape(32, 1)
    s = P.Pages(4, 4, 8, 4, [pool])
    assert s.extend([0, 1], [0, 0], [6, 4]) == ([2, 1], 0)
    assert s.table[0].tolist() == [0, 1, -1, -1] and s.table[1, 0] == 2
    assert s.fork([0, 0], [2, 3], [6, 8]) == ([1, 0], 0)
    assert s.table[2].tolist() == [0, 3, -1, -1] and s.table[3].tolist() == [0, 1, -1, -1]
    assert s.refs.tolist() == [3, 2, 1, 1, 0, 0, 0, 0]
    assert pool[12:14, 0].tolist() == [4, 5] and pool[14, 0] == 14
    assert s.extend([1, 0], [4, 6], [16, 16]) == ([3, -1], P.NOPAGE)  # 3 + 2 pages of 4
    s.check()
    assert s.release([0, 0, 9]) == P.TOKEN
    assert s.refs.tolist() == [2, 1, 1, 1, 1, 1, 1, 0]
    s.release([1], [1], [3])
    assert s.free == [7, 5, 4]
    s.compact()
    assert s.table[1].tolist() == [2, -1, -1, 4] and s.free == [7, 6, 5]
    s.check()


def test_row_and_attention_refusals_without_gpu():
    import hierarchical_sparse_attention_gb300 as hs
    A = 1 << 20  # an aligned stand-in address: nothing is launched in these calls
    rows = dict(n=4, kv=A, stride=576, rows=A, scale=1.0, pool=A, total=100, err=A)

    def pack(**kw):
        a = dict(rows, **kw)
        hs.hs_fp4_pack_rows(a["n"], a["kv"], a["stride"], a["rows"], a["scale"], a["pool"], a["total"], a["err"])

    def unpack(**kw):
        a = dict(rows, **kw)
        hs.hs_fp4_unpack_rows(a["n"], a["pool"], a["total"], a["rows"], a["scale"], a["kv"], a["stride"], a["err"])

    bad_scale = [dict(scale=x) for x in (0.0, -1.0, 3.0, math.nan, math.inf, 2.0 ** 33, 2.0 ** -33)]
    for kw in [dict(n=-1), dict(kv=None), dict(kv=A + 8), dict(stride=575), dict(stride=580), dict(rows=None),
               dict(pool=None), dict(pool=A + 8), dict(total=0), dict(err=None)] + bad_scale:
        for call in (pack, unpack):
            with pytest.raises(hs.HsError) as e:
                call(**kw)
            assert e.value.status == hs.HS_ERR_INVALID_ARG, kw
    pack(n=0, kv=None, rows=None, pool=None, err=None)
    unpack(n=0, kv=None, rows=None, pool=None, err=None)

    ws = hs.hs_fp4_mla_workspace_bytes
    assert ws(4, 128, 1, 1) == 0 and ws(4, 128, 2, 3) > 0
    for bad in ((0, 128, 1, 2), (4, 0, 1, 2), (4, 129, 1, 2), (4, 128, 0, 2), (4, 128, 9, 2), (4, 128, 1, 0), (4, 128, 1, 17)):
        assert ws(*bad) == 0
    good = dict(R=2, H=16, Q=1, splits=2, q=A, pool=A, total=100, sm=0.1, g=1.0, o=A, lse=A, ws=A, wsb=ws(2, 16, 2, 2), err=A,
                K=64, table=A, lens=A, W=8, sinks=1, page=16, mp=8)

    def sparse(**kw):
        a = dict(good, **kw)
        hs.hs_fp4_sparse_mla_decode(a["R"], a["H"], a["K"], a["splits"], a["q"], a["pool"], a["total"], a["table"], a["sm"],
                                    a["g"], a["o"], a["lse"], a["ws"], a["wsb"], a["err"])

    def window(**kw):
        a = dict(good, **kw)
        hs.hs_fp4_window_mla_decode(a["R"], a["H"], a["Q"], a["W"], a["sinks"], a["splits"], a["q"], a["pool"], a["total"],
                                    a["page"], a["mp"], a["lens"], a["table"], a["sm"], a["g"], a["o"], a["lse"], a["ws"],
                                    a["wsb"], a["err"])

    both = [dict(R=-1), dict(R=(1 << 20) + 1), dict(H=0), dict(H=129), dict(splits=0), dict(splits=17), dict(q=None), dict(q=A + 8),
            dict(pool=None), dict(pool=A + 8), dict(total=0), dict(total=1 << 31), dict(sm=math.inf), dict(sm=math.nan),
            dict(g=3.0), dict(o=None), dict(o=A + 4), dict(lse=None), dict(ws=None), dict(ws=A + 8), dict(wsb=15), dict(err=None),
            dict(table=None)]
    for call, kws in ((sparse, both + [dict(K=0), dict(K=hs.HS_MAX_TOP_K + 1)]),
                      (window, both + [dict(Q=0), dict(Q=9), dict(W=0), dict(sinks=-1), dict(page=0), dict(mp=0), dict(lens=None)])):
        for kw in kws:
            with pytest.raises(hs.HsError) as e:
                call(**kw)
            assert e.value.status == hs.HS_ERR_INVALID_ARG, kw
        call(R=0, q=None, pool=None, table=None, lens=None, o=None, lse=None, ws=None, wsb=0, err=None)


def test_page_refusals_without_gpu():
    import hierarchical_sparse_attention_gb300 as hs
    A = 1 << 20
    wsb = hs.hs_pages_workspace_bytes(4, 100)
    assert wsb > 0
    for bad in ((0, 100), (hs.HS_MAX_PAGE_REQUESTS + 1, 100), (4, 0)):
        assert hs.hs_pages_workspace_bytes(*bad) == 0

    def pool(**kw):
        a = dict(pools=[A, A], R=4, mp=8, n=100, ps=16, rb=416, table=A, refs=A, free=A, count=A, ws=A, wsb=wsb, err=A)
        a.update(kw)
        return hs.make_page_pool(a["pools"], a["R"], a["mp"], a["n"], a["ps"], a["rb"], a["table"], a["refs"], a["free"],
                                 a["count"], a["ws"], a["wsb"], a["err"])

    calls = [lambda p: hs.hs_pages_init(p), lambda p: hs.hs_pages_extend(p, 1, A, A, A), lambda p: hs.hs_pages_fork(p, 1, A, A, A),
             lambda p: hs.hs_pages_free(p, 1, A), lambda p: hs.hs_pages_compact(p)]
    for kw in (dict(pools=[A, None]), dict(R=0), dict(R=hs.HS_MAX_PAGE_REQUESTS + 1), dict(mp=0), dict(n=0), dict(ps=0), dict(rb=0),
               dict(n=1 << 27, wsb=1 << 40), dict(mp=1 << 27), dict(table=None), dict(refs=None), dict(free=None),
               dict(count=None), dict(ws=None), dict(ws=A + 8), dict(wsb=wsb - 1), dict(err=None)):
        for call in calls:
            with pytest.raises(hs.HsError) as e:
                call(pool(**kw))
            assert e.value.status == hs.HS_ERR_INVALID_ARG, kw
    for call in calls:
        with pytest.raises(hs.HsError):
            call(None)
    p = pool()
    for call in (lambda: hs.hs_pages_extend(p, -1, A, A, A), lambda: hs.hs_pages_extend(p, 1, None, A, A),
                 lambda: hs.hs_pages_extend(p, 1, A, None, A), lambda: hs.hs_pages_extend(p, 1, A, A, None),
                 lambda: hs.hs_pages_fork(p, 5, A, A, A), lambda: hs.hs_pages_fork(p, 1, None, A, A),
                 lambda: hs.hs_pages_fork(p, 1, A, None, A), lambda: hs.hs_pages_fork(p, 1, A, A, None),
                 lambda: hs.hs_pages_free(p, -1, A), lambda: hs.hs_pages_free(p, 1, None)):
        with pytest.raises(hs.HsError) as e:
            call()
        assert e.value.status == hs.HS_ERR_INVALID_ARG
    hs.hs_pages_extend(p, 0, None, None, None)
    hs.hs_pages_fork(p, 0, None, None, None)
    hs.hs_pages_free(p, 0, None)
    with pytest.raises(ValueError):
        pool(pools=[])
    with pytest.raises(ValueError):
        pool(pools=[A] * 9)


def test_tensors_of_another_kind_are_refused_without_gpu():
    torch = pytest.importorskip("torch")
    import hierarchical_sparse_attention_gb300 as hs
    A = 1 << 20
    host = torch.zeros(4, 576, dtype=torch.int16)
    with pytest.raises(ValueError):
        hs.hs_fp4_pack_rows(4, host, 576, A, 1.0, A, 100, A)
    with pytest.raises(ValueError):
        hs.hs_fp4_pack_rows(4, host, 640, A, 1.0, A, 100, A)
    with pytest.raises(ValueError):
        hs.make_page_pool([host], 4, 8, 100, 16, 416, A, A, A, A, A, 1 << 20, A)
    assert ctypes.sizeof(hs.hs_page_pool) == 6 * 4 + 8 * 8 + 6 * 8 + 8
