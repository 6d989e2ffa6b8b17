"""CPU ORACLE of a step with several new tokens of a sequence (the batch's plan, fp8 MLA rows, attention
of the chunks) -- TEST INFRASTRUCTURE ONLY. Plain numpy, attention in float64.

A row is 656 B: 512 e4m3 codes, 4 fp32 scales (one per 128 dims), 64 bf16 RoPE values; latent = e4m3 x scale.
"""
from __future__ import annotations

import numpy as np

from .fp4_mla import attend, nearest_code
from .sparse_mla import bf16_decode, e4m3_decode

ROW, LATENT, ROPE, BLOCK = 656, 512, 64, 128
DIMS = LATENT + ROPE
E4M3 = e4m3_decode(np.arange(127))  # 0 .. 448, ascending
TOKEN, DUP, DEVROW, SEQLEN, FULL = 1, 2, 16, 32, 512


def plan(requests, old_lens, new_lens, table, page, pool_rows, max_tokens, max_blocks=None):
    """Entry by entry: dict of the call's outputs, and its flags."""
    n, (num_requests, max_pages) = len(requests), table.shape
    out = {"token_offsets": np.zeros(n + 1, np.int32), "seq_lens": np.zeros(n, np.int32)}
    for k in ("entries", "positions", "rows"):
        out[k] = np.full(max_tokens, -1, np.int32)
    if max_blocks is not None:
        out["block_tables"] = np.full((n, max_blocks), -1, np.int32)
    flags, asked, at = 0, 0, 0
    for i in range(n):
        r, a, b = int(requests[i]), int(old_lens[i]), int(new_lens[i])
        ok = r >= 0
        if ok and r >= num_requests:
            ok, flags = False, flags | TOKEN
        elif ok and sum(int(x) == r for x in requests) > 1:
            ok, flags = False, flags | DUP
        elif ok and (a < 0 or b < a or b > page * min(max_pages, max_pages if max_blocks is None else max_blocks)):
            ok, flags = False, flags | SEQLEN
        if ok:
            asked += b - a
            if b > a and asked > max_tokens:
                ok, flags = False, flags | FULL
        if ok:
            out["seq_lens"][i] = b
            for p in range(a, b):
                pg = int(table[r, p // page])
                row = pg * page + p % page
                if pg < 0 or row >= pool_rows:
                    row, flags = -1, flags | DEVROW
                out["entries"][at], out["positions"][at], out["rows"][at] = i, p, row
                at += 1
            if max_blocks is not None:
                held = -(-b // page)
                out["block_tables"][i, :held] = table[r, :held]
        out["token_offsets"][i + 1] = at
    return out, flags


def pack(kv_bits, weight_bits=None, eps=0.0, positions=None, rope=None):
    """bf16 bit patterns [n, 576] -> (rows' codes and scales [n, 528] as bytes, RoPE values [n, 64] in 64 bits)."""
    n = kv_bits.shape[0]
    x = bf16_decode(kv_bits[:, :LATENT])
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        y = x
        if weight_bits is not None:
            y = x * bf16_decode(weight_bits)[None] / np.sqrt(np.square(x).mean(1, keepdims=True) + np.float64(np.float32(eps)))
            y[~np.isfinite(x).all(1)] = np.nan
    y = y.reshape(n, -1, BLOCK)
    bad = ~np.isfinite(y).all(-1)
    y = np.where(bad[..., None], 0.0, y)
    mant, e = np.frexp(np.abs(y).max(-1))  # top = mant 2^e; 448 = 0.875 x 2^9
    k = np.maximum(np.where(mant > 0.875, e - 8, e - 9), -126)
    k = np.where(mant == 0, -126, k)
    q = np.ldexp(y, -k[..., None])
    code = nearest_code(np.abs(q), E4M3) | np.where(np.signbit(q), 128, 0)
    code[bad] = 0
    scale = np.where(bad, np.nan, np.ldexp(1.0, k)).astype(np.float32)
    out = np.empty((n, LATENT + 16), np.uint8)
    out[:, :LATENT] = code.reshape(n, LATENT)
    out[:, LATENT:] = np.ascontiguousarray(scale).view(np.uint8)
    r = bf16_decode(kv_bits[:, LATENT:])
    if rope is not None:
        cs = rope[positions].astype(np.float64)
        a, b, c, s = r[:, 0::2], r[:, 1::2], cs[:, :ROPE // 2], cs[:, ROPE // 2:]
        r = np.stack((a * c - b * s, a * s + b * c), -1).reshape(n, ROPE)
    return out, r


def unpack(rec):
    """Rows [n, 656] -> (latent [n, 512], rope [n, 64]) in 64 bits."""
    scale = np.ascontiguousarray(rec[:, LATENT:LATENT + 16]).view(np.float32).astype(np.float64)
    with np.errstate(invalid="ignore"):
        lat = e4m3_decode(rec[:, :LATENT]) * np.repeat(scale, BLOCK, axis=1)
    return lat, bf16_decode(np.ascontiguousarray(rec[:, LATENT + 16:]).view("<u2"))


def chunk_entry(q, seq, nq, pages, page, pool, sm):
    """One entry: q [nq, h, 576] in 64 bits, its page numbers, the pool's bytes. Returns o [nq, h, 512], lse [nq, h] and,
    for error bounds, A = sum_j p_j |latent_j|, B = the largest sm sum |q k| of a head, C = sum_j |latent_j| of the rows seen."""
    h = q.shape[1]
    o, A, C = (np.zeros((nq, h, LATENT)) for _ in range(3))
    lse, B = np.full((nq, h), -np.inf), np.zeros((nq, h))
    t = np.arange(max(seq, 0))
    pg = pages[t // page].astype(np.int64)
    rows = pg * page + t % page
    there = (pg >= 0) & (rows < pool.shape[0])
    lat, rope = unpack(pool[np.where(there, rows, 0)])
    for i in range(nq):
        see = there & (t <= seq - nq + i)
        o[i], lse[i], A[i], B[i] = attend(q[i], lat[see], rope[see], sm)
        C[i] = np.abs(lat[see]).sum(0)
    return o, lse, A, B, C
