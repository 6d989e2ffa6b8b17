"""The oracle of steps with several new tokens, against worked examples and closed forms (no GPU)."""
import numpy as np
import pytest

from oracle import chunk as C
from oracle.sparse_mla import bf16_decode


def bits(x):
    torch = pytest.importorskip("torch")
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def test_a_plan_worked_by_hand():
    """Pages of 4 tokens: request 2 goes from 3 to 6 tokens, request 0 from 0 to 1, an entry is padding, and the last one
    of 3 tokens finds room for 2."""
    table = np.array([[7, -1, -1], [-1, -1, -1], [5, 2, -1], [1, 3, -1]], np.int32)
    out, flags = C.plan([2, -1, 0, 3], [3, 9, 0, 4], [6, 9, 1, 7], table, 4, 100, 6, 2)
    assert out["token_offsets"].tolist() == [0, 3, 3, 4, 4] and out["seq_lens"].tolist() == [6, 0, 1, 0]
    assert out["entries"].tolist() == [0, 0, 0, 2, -1, -1] and out["positions"].tolist() == [3, 4, 5, 0, -1, -1]
    assert out["rows"].tolist() == [23, 8, 9, 28, -1, -1]
    assert out["block_tables"].tolist() == [[5, 2], [-1, -1], [7, -1], [-1, -1]] and flags == C.FULL


def test_a_plan_refuses_entries():
    table = np.arange(12, dtype=np.int32).reshape(4, 3)
    out, flags = C.plan([1, 4, 1, 0, 2, 3], [0, 0, 0, 2, 0, -1], [1, 1, 1, 1, 13, 2], table, 4, 100, 50)
    assert out["token_offsets"].tolist() == [0] * 7 and flags == C.TOKEN | C.DUP | C.SEQLEN
    out, flags = C.plan([0, 1], [0, 0], [2, 2], np.array([[-1], [25]], np.int32), 4, 101, 9)
    assert out["rows"].tolist() == [-1, -1, 100, -1, -1, -1, -1, -1, -1] and flags == C.DEVROW


def test_rows_of_exact_values():
    """Values that e4m3 holds come back as they are; 448 is the largest of a scale, so that 15 and 452 take the next ones."""
    kv = np.zeros((3, 576))
    kv[0, :128] = np.arange(128) % 16
    kv[0, 128:256] = -448 * 2.0 ** -5
    kv[0, 256] = 452.0  # over a scale of 2: 226, whose nearest e4m3 value is 224
    kv[0, 512:] = np.arange(64)
    rec, rope = C.pack(bits(kv))
    lat, _ = C.unpack(np.concatenate((rec, np.zeros((3, 128), np.uint8)), 1))
    assert np.array_equal(lat[0, :256], kv[0, :256]) and np.array_equal(rope, kv[:, 512:])
    scale = rec[:, 512:].copy().view(np.float32)
    assert scale[0].tolist() == [2.0 ** -4, 2.0 ** -5, 2.0, 2.0 ** -126] and lat[0, 256] == 448.0


def test_the_norm_and_the_rotation():
    rng = np.random.default_rng(0)
    kv, w = rng.standard_normal((4, 576)) * 3, 1 + rng.standard_normal(512) * 0.1
    kb, wb = bits(kv), bits(w)
    ang = rng.uniform(0, 6, (9, 32))
    table = np.concatenate((np.cos(ang), np.sin(ang)), 1).astype(np.float32)
    rec, rope = C.pack(kb, wb, 1e-6, np.array([0, 3, 8, 8]), table)
    x = bf16_decode(kb)
    y = x[:, :512] * bf16_decode(wb) / np.sqrt((x[:, :512] ** 2).mean(1, keepdims=True) + 1e-6)
    lat, _ = C.unpack(np.concatenate((rec, np.zeros((4, 128), np.uint8)), 1))
    # a step of e4m3 is at most 2^-3 of the value, or 2^-9 of the scale below the normal range; rounding is off by half a step
    assert (np.abs(lat - y) <= np.maximum(np.abs(y) / 16, 2.0 ** -10 * np.repeat(rec[:, 512:].copy().view(np.float32), 128, 1))).all()
    # a rotation keeps lengths (the table's cosines and sines are off by up to 2^-25)
    n0, n1 = np.hypot(x[:, 512::2], x[:, 513::2]), np.hypot(rope[:, 0::2], rope[:, 1::2])
    assert np.allclose(n0, n1, rtol=1e-6)
    bad = kb.copy()
    bad[1, 7] = 0x7F80
    assert np.isnan(C.unpack(np.concatenate((C.pack(bad, wb, 1e-6)[0], np.zeros((4, 128), np.uint8)), 1))[0][1]).all()


def test_attention_closed_forms():
    rng = np.random.default_rng(1)
    kv = rng.standard_normal((12, 576))
    rec = np.concatenate((C.pack(bits(kv))[0], bits(kv[:, 512:]).view(np.uint8)), 1)
    lat, rope = C.unpack(rec)
    pages = np.array([2, 0, 1], np.int32)  # of 4 rows
    order = np.r_[8:12, 0:4, 4:8]
    o, lse, *_ = C.chunk_entry(np.zeros((3, 2, 576)), 7, 3, pages, 4, rec, 0.3)
    for i in range(3):  # a query of zeros averages what it sees
        assert np.allclose(o[i], lat[order[:5 + i]].mean(0)) and np.allclose(lse[i], np.log(5 + i))
    q = rng.standard_normal((1, 1, 576))
    o, lse, *_ = C.chunk_entry(q, 1, 1, pages, 4, rec, 0.3)  # one row: its latent, its score
    assert np.allclose(o[0, 0], lat[8]) and np.allclose(lse, 0.3 * (q[0, 0, :512] @ lat[8] + q[0, 0, 512:] @ rope[8]))
    o, lse, *_ = C.chunk_entry(np.ones((3, 1, 576)), 2, 3, pages, 4, rec, 0.3)  # the first query stands before the sequence
    assert (o[0] == 0).all() and lse[0] == -np.inf and np.isfinite(lse[1:]).all()
    o, lse, *_ = C.chunk_entry(np.zeros((1, 1, 576)), 7, 1, np.array([-1, 3, 1], np.int32), 4, rec, 0.3)  # pages that are not there
    assert (o == 0).all() and lse == -np.inf
