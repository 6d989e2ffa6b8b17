"""Cases of the operators of a step with several new tokens of a sequence, their plain forms, and what they have to compute.

A step's batch is a list of entries (request, tokens that it held before, tokens that it holds with the new ones). Rows are
one token's MLA key/value in 656 bytes: 512 e4m3 codes, 4 fp32 scales (one per 128 codes; the rows written here have powers
of two) and 64 bf16 RoPE values, in pages of a pool.

kind "plan":   hs_batch_plan, the batch's offsets, positions, pool rows and block tables from the entries and the page table
kind "rows":   hs_fp8_pack_rows normalises, rotates and quantises new tokens into their rows, hs_fp8_unpack_rows reads rows back
kind "chunk":  hs_chunk_mla, attention of the entries' new tokens over the pages of their sequences, causal
"""
import math

import numpy as np
import torch

own = False

ROW, LATENT, ROPE, DIMS, BLOCK = 656, 512, 64, 576, 128
SM_SCALE = 1.0 / math.sqrt(192.0)
EPS = 1e-6


def listed():
    return [
        # a decode step of the 32-request DSA workload: one new token each
        {"name": "plan_step", "kind": "plan", "entries": 32, "pad": 0, "new_lo": 1, "new_hi": 1, "ctx_lo": 100000, "ctx_hi": 131000, "page": 64, "max_pages": 2048, "slots": 48,
         "room": 0},
        # a large step: decodes, chunks and padding entries, with a block table for each
        {"name": "plan_chunks", "kind": "plan", "entries": 1024, "pad": 60, "new_lo": 1, "new_hi": 96, "ctx_lo": 0, "ctx_hi": 65536, "page": 64, "max_pages": 1040, "slots": 1100,
         "room": 3000},
        # the rows of that decode step's tokens
        {"name": "rows8_step", "kind": "rows", "n": 32, "m": 32, "pool_rows": 4096, "stride": 576},
        # a prefill chunk's rows, and twice as many read back
        {"name": "rows8_prefill", "kind": "rows", "n": 32768, "m": 65536, "pool_rows": 131072, "stride": 640},
        # the tiny workload's two sequences, a token each, the 16 heads of one tensor-parallel rank
        {"name": "chunk_tiny", "kind": "chunk", "heads": 16, "ones": 2, "chunks": 0, "pad": 0, "new_lo": 1, "new_hi": 1, "ctx_lo": 100, "ctx_hi": 8192, "page": 64, "room": 0},
        # verify steps of speculative decoding, ragged, on one rank, some entries padded
        {"name": "chunk_verify", "kind": "chunk", "heads": 16, "ones": 0, "chunks": 64, "pad": 4, "new_lo": 2, "new_hi": 4, "ctx_lo": 10, "ctx_hi": 8192, "page": 64, "room": 9},
        # a decode step with all heads
        {"name": "chunk_decode", "kind": "chunk", "heads": 128, "ones": 32, "chunks": 0, "pad": 0, "new_lo": 1, "new_hi": 1, "ctx_lo": 500, "ctx_hi": 4095, "page": 64, "room": 0},
        # a first chunk: nothing in the cache before it
        {"name": "chunk_first", "kind": "chunk", "heads": 128, "ones": 0, "chunks": 1, "pad": 0, "new_lo": 2048, "new_hi": 2048, "ctx_lo": 0, "ctx_hi": 0, "page": 64, "room": 0},
        # a mixed step: decodes beside two chunks, pages that end inside tiles
        {"name": "chunk_mixed", "kind": "chunk", "heads": 64, "ones": 30, "chunks": 2, "pad": 0, "new_lo": 400, "new_hi": 700, "ctx_lo": 300, "ctx_hi": 12000, "page": 48, "room": 100},
        # chunks of several sequences on one rank
        {"name": "chunk_rank", "kind": "chunk", "heads": 16, "ones": 0, "chunks": 8, "pad": 0, "new_lo": 512, "new_hi": 512, "ctx_lo": 6000, "ctx_hi": 8191, "page": 64, "room": 0},
        # a chunk far into a long sequence
        {"name": "chunk_long", "kind": "chunk", "heads": 128, "ones": 0, "chunks": 1, "pad": 0, "new_lo": 256, "new_hi": 256, "ctx_lo": 48000, "ctx_hi": 48000, "page": 64, "room": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


MOST_FLOPS = 3.2e12  # of a drawn attention case (the largest listed one: 3.4e12)


def draw(rng):
    kind = rng.choice(["plan", "rows", "chunk", "chunk", "chunk", "chunk"])
    page = rng.choice([1, 16, 48, 64, 64, 128])
    if kind == "plan":
        n, new = _log(rng, 1, 1024), _log(rng, 1, 96)
        ctx = _log(rng, 1, 131000 if n < 400 else 60000)
        return {"kind": kind, "entries": n, "pad": rng.randint(0, n // 8), "new_lo": rng.choice([0, 1, new]), "new_hi": new, "ctx_lo": rng.randint(0, ctx), "ctx_hi": ctx, "page": max(16, page),
                "max_pages": -(-(ctx + new) // max(16, page)) + rng.randint(0, 9), "slots": n + rng.randint(0, 50), "room": rng.choice([0, _log(rng, 1, 3000)])}
    if kind == "rows":
        n, m = _log(rng, 1, 32768), _log(rng, 1, 65536)
        return {"kind": kind, "n": n, "m": m, "pool_rows": max(n, m) + _log(rng, 1, 50000), "stride": 576 + 8 * rng.choice([0, 0, 1, 8, 64])}
    heads = rng.choice([128, 64, 16, _log(rng, 1, 128)])
    ones, chunks = rng.choice([0, _log(rng, 1, 64)]), rng.choice([0, 1, _log(rng, 1, 64)])
    if ones + chunks == 0:
        ones = 1
    ctx = _log(rng, 1, 48000)
    most = max(1.0, MOST_FLOPS / (2.0 * (DIMS + LATENT) * heads * ctx) - ones)
    new = _log(rng, 1, int(max(1, min(2048, most / max(1, chunks)))))
    while (ones + chunks) * (ctx + new) > 500000 or (ones + chunks * new) * (ctx + new) * heads * 2.0 * (DIMS + LATENT) > MOST_FLOPS:
        ctx = ctx // 2 + 1
        new = new // 2 + 1
        ones, chunks = ones // 2 + (chunks == 0), chunks // 2 + (chunks == 1)
    return {"kind": kind, "heads": heads, "ones": ones, "chunks": chunks, "pad": rng.randint(0, 3), "new_lo": rng.randint(1, new), "new_hi": new, "ctx_lo": rng.choice([0, ctx // 2, ctx]),
            "ctx_hi": ctx, "page": page, "room": rng.choice([0, 1, _log(rng, 1, 200)])}


def work(case):
    """Each input read once and each output written once; the two matrix products of attention."""
    k = case["kind"]
    if k == "plan":
        b = _batch(case, 0)
        blocks = int((-(-b["new"] // case["page"])).sum())  # table entries that hold a page
        n = case["entries"]
        return {"bytes": 12 * n + 4 * (2 * n + 1) + 12 * b["max_tokens"] + 4 * blocks + 4 * n * case["max_pages"], "flops": 0}
    if k == "rows":
        return {"bytes": case["n"] * (DIMS * 2 + 8 + ROPE * 4 + ROW) + case["m"] * (ROW + 4 + DIMS * 2), "flops": case["n"] * (4 * LATENT + 3 * ROPE)}
    b = _batch(case, 0)
    t, new = (b["new"] - b["old"]).astype(np.float64), b["new"].astype(np.float64)
    seen = float((t * new - t * (t - 1) / 2).sum())
    rows, h = float(new.sum()), case["heads"]
    return {"bytes": rows * (ROW + 4 / case["page"]) + float(t.sum()) * h * (DIMS * 2 + LATENT * 2 + 4), "flops": 2 * seen * h * (DIMS + LATENT)}


# ---------------------------------------------------------------- inputs


def _batch(case, seed):
    """The entries of a step on the host: tokens before (old) and with the new ones (new), in batch order."""
    g = np.random.default_rng([seed, 21])
    if case["kind"] == "plan":
        n, live = case["entries"], case["entries"] - case["pad"]
        old, new = np.zeros(n, dtype=np.int64), np.zeros(n, dtype=np.int64)
        old[:live] = g.integers(case["ctx_lo"], case["ctx_hi"] + 1, size=live)
        new[:live] = old[:live] + np.linspace(case["new_lo"], case["new_hi"], live).astype(np.int64)[g.permutation(live)]
    else:
        n, ones, live = case["ones"] + case["chunks"] + case["pad"], case["ones"], case["ones"] + case["chunks"]
        # evenly spread lengths in a random order, so that every seed has the same number of tokens
        old = np.zeros(n, dtype=np.int64)
        old[:live] = np.linspace(case["ctx_lo"], case["ctx_hi"], live).astype(np.int64)[g.permutation(live)]
        new = old.copy()
        new[:ones] += 1
        new[ones:live] += np.linspace(case["new_lo"], case["new_hi"], live - ones).astype(np.int64)[g.permutation(live - ones)]
    total = int((new - old).sum())
    return {"old": old.astype(np.int64), "new": new.astype(np.int64), "live": live, "max_tokens": max(1, total + case["room"])}


def _new_tokens(gen, n):
    """bf16 latents before their norm (a few loud dims) and RoPE values of n tokens, on the GPU."""
    gain = torch.ones(DIMS, device="cuda")
    gain[:LATENT:37] = 6.0
    gain[5:LATENT:11] = 0.05
    return (torch.randn(n, DIMS, generator=gen, device="cuda") * gain).to(torch.bfloat16)


def _pool(gen, rows):
    pool = torch.empty(rows, ROW, dtype=torch.uint8, device="cuda")
    for at in range(0, rows, 65536):
        kv = _new_tokens(gen, min(65536, rows - at)).float()
        y = kv[:, :LATENT].view(-1, LATENT // BLOCK, BLOCK)
        scale = torch.exp2(torch.ceil(torch.log2(y.abs().amax(-1, keepdim=True) / 448.0)))
        rec = pool[at:at + 65536]
        rec[:, :LATENT] = (y / scale).to(torch.float8_e4m3fn).view(torch.uint8).view(-1, LATENT)
        rec[:, LATENT:LATENT + 16] = scale.view(-1, 4).contiguous().view(torch.uint8)
        rec[:, LATENT + 16:] = kv[:, LATENT:].to(torch.bfloat16).contiguous().view(torch.uint8)
    return pool


def _tables(b, page, max_pages, slots, seed):
    """A page table with random pages for every entry's tokens, and the entries' requests (padding: -1)."""
    g = np.random.default_rng([seed, 22])
    n = b["new"].size
    requests = g.permutation(slots)[:n].astype(np.int32)
    requests[b["live"]:] = -1
    held = -(-b["new"] // page)
    table = np.full((slots, max_pages), -1, dtype=np.int32)
    perm = g.permutation(int(held.sum()) + 7).astype(np.int32)
    at = 0
    for i in range(b["live"]):
        table[requests[i], :held[i]] = perm[at:at + held[i]]
        at += int(held[i])
    return table, requests, perm.size


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    st = {"case": dict(case), "keep": {}}
    if case["kind"] == "plan":
        b = _batch(case, seed)
        table, requests, pages = _tables(b, case["page"], case["max_pages"], case["slots"], seed)
        st["max_tokens"], st["pool_rows"] = b["max_tokens"], pages * case["page"]
        for name, x in (("table", table), ("requests", requests), ("old", b["old"]), ("new", b["new"])):
            st[name] = torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()
        return st
    if case["kind"] == "rows":
        n, m, total = case["n"], case["m"], case["pool_rows"]
        wide = torch.randn(n, case["stride"], generator=gen, device="cuda").to(torch.bfloat16)
        wide[:, :DIMS] = _new_tokens(gen, n)
        st["kv"] = wide[:, :DIMS]  # a slice of a wider projection
        order = torch.randperm(total, generator=gen, device="cuda")
        rows = order[:n].to(torch.int32)
        rows[torch.rand(n, generator=gen, device="cuda") < 0.02] = -1  # padding tokens of the batch
        st["rows"] = rows
        st["positions"] = torch.randint(0, 131072, (n,), generator=gen, device="cuda", dtype=torch.int32)
        st["weight"] = (1.0 + 0.3 * torch.randn(LATENT, generator=gen, device="cuda")).to(torch.bfloat16)
        angle = torch.arange(131072, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, ROPE, 2, device="cuda", dtype=torch.float64) / ROPE)
        st["rope"] = torch.cat((torch.cos(angle), torch.sin(angle)), -1).float()
        st["pool"] = _pool(gen, total)
        back = order[torch.randperm(max(n, m), generator=gen, device="cuda")[:m]].to(torch.int32)
        back[torch.rand(m, generator=gen, device="cuda") < 0.02] = -1
        st["back"] = back
        return st
    b = _batch(case, seed)
    n, page = b["new"].size, case["page"]
    max_pages = max(1, int((-(-b["new"] // page)).max()))
    table, requests, pages = _tables(b, page, max_pages, n, seed)
    tables = np.full((n, max_pages), -1, dtype=np.int32)  # by entry
    tables[requests >= 0] = table[requests[requests >= 0]]
    offsets = np.concatenate([[0], np.cumsum(b["new"] - b["old"])])
    st["max_tokens"], st["offsets_host"], st["lens_host"] = b["max_tokens"], offsets, b["new"]
    for name, x in (("tables", tables), ("offsets", offsets), ("lens", b["new"])):
        st[name] = torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()
    st["pool"] = _pool(gen, pages * page)
    st["q"] = torch.randn(b["max_tokens"], case["heads"], DIMS, generator=gen, device="cuda").to(torch.bfloat16)
    st["o"] = torch.zeros(b["max_tokens"], case["heads"], LATENT, dtype=torch.bfloat16, device="cuda")
    st["lse"] = torch.zeros(b["max_tokens"], case["heads"], dtype=torch.float32, device="cuda")
    return st


# ---------------------------------------------------------------- plain forms


def _plain_plan(st):
    c, dev = st["case"], st["table"].device
    n, ps, room = st["requests"].numel(), c["page"], st["max_tokens"]
    live = st["requests"] >= 0
    old, new = st["old"].long(), st["new"].long()
    count = torch.where(live, new - old, torch.zeros_like(old))
    lens = torch.where(live, new, torch.zeros_like(new))
    offsets = torch.zeros(n + 1, dtype=torch.int64, device=dev)
    offsets[1:] = torch.cumsum(count, 0)
    slot = torch.arange(room, device=dev)
    entry = torch.searchsorted(offsets[1:], slot, right=True)
    there = entry < n
    e = entry.clamp(max=n - 1)
    at = old[e] + slot - offsets[e]
    tables = torch.where(live[:, None], st["table"][st["requests"].clamp(min=0).long()], torch.full((), -1, dtype=torch.int32, device=dev))
    held = torch.arange(c["max_pages"], device=dev)[None] < ((lens + ps - 1) // ps)[:, None]
    tables = torch.where(held, tables, torch.full_like(tables, -1))
    page = tables[e, (at // ps).clamp(0, c["max_pages"] - 1)].long()
    none = torch.full_like(slot, -1)
    rows = torch.where(there & (page >= 0), page * ps + at % ps, none)
    return {"offsets": offsets.int(), "lens": lens.int(), "entries": torch.where(there, entry, none).int(), "positions": torch.where(there, at, none).int(),
            "rows": rows.int(), "tables": tables}


def _round_e4m3(x):
    """The nearest e4m3 values (halfway: the even code) of values up to 448, in 64 bits."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return torch.round(x / step) * step


def _plain_rows(st):
    rows, back, total = st["rows"], st["back"], st["pool"].shape[0]
    x = st["kv"][:, :LATENT].double()  # (64 bits: values next to a border between two codes)
    y = x * st["weight"].double() / torch.sqrt((x * x).mean(-1, keepdim=True) + float(np.float32(EPS)))
    y = y.view(-1, LATENT // BLOCK, BLOCK)
    mant, e = torch.frexp(y.abs().amax(-1, keepdim=True))  # top = mant 2^e, and 448 = 0.875 x 2^9
    scale = torch.exp2((e - 9 + (mant > 0.875)).double())
    code = _round_e4m3(y / scale).view(-1, LATENT)
    r = st["kv"][:, LATENT:].float()
    cs = st["rope"][st["positions"].long()].double()
    a, b, cos, sin = r[:, 0::2].double(), r[:, 1::2].double(), cs[:, :ROPE // 2], cs[:, ROPE // 2:]
    turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(1).to(torch.bfloat16)
    rec = torch.empty(rows.numel(), ROW, dtype=torch.uint8, device=rows.device)
    rec[:, :LATENT] = code.float().to(torch.float8_e4m3fn).view(torch.uint8)
    rec[:, LATENT:LATENT + 16] = scale.float().view(-1, 4).contiguous().view(torch.uint8)
    rec[:, LATENT + 16:] = turned.view(torch.uint8)
    ok = rows >= 0
    st["pool"][rows[ok].long()] = rec[ok]
    live = (back >= 0) & (back < total)
    lat, rope = _values(st["pool"][back.clamp(min=0).long()])
    return torch.where(live[:, None], torch.cat((lat, rope), -1), torch.zeros((), device=rows.device)).to(torch.bfloat16)


def _values(rec):
    """(latent [..., 512], rope [..., 64]) in 32 bits of rows' bytes [..., 656]."""
    code = rec[..., :LATENT].contiguous().view(torch.float8_e4m3fn).float()
    scale = rec[..., LATENT:LATENT + 16].contiguous().view(torch.float32)
    lat = (code.view(*code.shape[:-1], LATENT // BLOCK, BLOCK) * scale[..., None]).flatten(-2)
    return lat, rec[..., LATENT + 16:].contiguous().view(torch.bfloat16).float()


def _plain_chunk(st):
    """Entries with about as many new tokens are computed together, padded, in pieces whose scores take up to about 1.2 GB."""
    ps, h, q, dev = st["case"]["page"], st["case"]["heads"], st["q"], st["q"].device
    counts = np.diff(st["offsets_host"])
    o, lse = torch.zeros_like(st["o"]), torch.zeros_like(st["lse"])
    for size in np.unique(np.frexp(counts[counts > 0] - 0.5)[1]):
        group = np.flatnonzero((counts > 0) & (np.frexp(counts - 0.5)[1] == size))
        longest, most = int(st["lens_host"][group].max()), int(counts[group].max())
        for part in np.array_split(group, -(-group.size * longest * max(h, 128) // 300000000)):
            at = torch.from_numpy(part).to(dev, non_blocking=True)
            t = torch.arange(longest, device=dev)
            page = st["tables"][at][:, t // ps].long()
            lat, rope = _values(st["pool"][page.clamp(min=0) * ps + t % ps])
            k = torch.cat((lat, rope), -1).transpose(1, 2)
            first, end, length = st["offsets"][at].long(), st["offsets"][at + 1].long(), st["lens"][at].long()
            step = max(1, 300000000 // (part.size * h * longest))
            for x in range(0, most, step):
                m = min(step, most - x)
                tok = first[:, None] + x + torch.arange(m, device=dev)
                there = tok < end[:, None]
                tok = torch.where(there, tok, first[:, None])
                s = torch.matmul(q[tok].float().view(part.size, m * h, DIMS), k).view(part.size, m, h, longest) * SM_SCALE
                see = (length - end)[:, None] + tok  # the last position that a token sees: its own
                s.masked_fill_((t > see[..., None])[:, :, None], -math.inf)
                top = s.amax(-1, keepdim=True)
                p = torch.exp(s - top)
                z = p.sum(-1, keepdim=True)
                y = torch.matmul(p.view(part.size, m * h, longest), lat).view(part.size, m, h, LATENT) / z
                o[tok[there]] = y[there].to(torch.bfloat16)
                lse[tok[there]] = (top + torch.log(z))[..., 0][there]
    return o, lse


# ---------------------------------------------------------------- the framework's calls


def _flags(keep):
    if "err" not in keep:
        keep["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return keep["err"]


def _own_plan(st, hs):
    c, n, room = st["case"], st["requests"].numel(), st["max_tokens"]
    ints = lambda *shape: torch.empty(*shape, dtype=torch.int32, device="cuda")
    out = {"offsets": ints(n + 1), "lens": ints(n), "entries": ints(room), "positions": ints(room), "rows": ints(room), "tables": ints(n, c["max_pages"])}
    hs.hs_batch_plan(n, st["requests"], st["old"], st["new"], c["slots"], st["table"], c["max_pages"], c["page"], st["pool_rows"], room, out["offsets"], out["lens"],
                     out["entries"], out["positions"], out["rows"], c["max_pages"], out["tables"], _flags(st["keep"]))
    return out


def _own_rows(st, hs):
    kv, pool, keep = st["kv"], st["pool"], st["keep"]
    out = torch.empty(st["back"].shape[0], DIMS, dtype=torch.bfloat16, device="cuda")
    hs.hs_fp8_pack_rows(kv.shape[0], kv, kv.stride(0), st["rows"], st["weight"], EPS, st["positions"], st["rope"], st["rope"].shape[0], pool, pool.shape[0], _flags(keep))
    hs.hs_fp8_unpack_rows(out.shape[0], pool, pool.shape[0], st["back"], out, DIMS, _flags(keep))
    return out


def _own_chunk(st, hs):
    c, q, pool, keep = st["case"], st["q"], st["pool"], st["keep"]
    n = st["lens"].numel()
    if "ws" not in keep:
        keep["kv"] = int((-(-st["lens_host"] // 64) * 64).sum())  # what the batch's sequences take, in whole blocks of 64 tokens
        keep["bytes"] = hs.hs_chunk_mla_workspace_bytes(n, c["heads"], st["max_tokens"], keep["kv"])
        keep["ws"] = torch.zeros(keep["bytes"], dtype=torch.uint8, device="cuda")
    hs.hs_chunk_mla(n, c["heads"], st["max_tokens"], st["offsets"], st["lens"], q, pool, pool.shape[0], c["page"], st["tables"].shape[1], st["tables"], SM_SCALE, st["o"], st["lse"],
                    keep["kv"], keep["ws"], keep["bytes"], _flags(keep))
    return st["o"], st["lse"]


def run(state):
    kind = state["case"]["kind"]
    if own:
        import hierarchical_sparse_attention_gb300 as hs

        return {"plan": _own_plan, "rows": _own_rows, "chunk": _own_chunk}[kind](state, hs)
    return {"plan": _plain_plan, "rows": _plain_rows, "chunk": _plain_chunk}[kind](state)


# ---------------------------------------------------------------- the definitions in 64 bits


def _exact_plan(case, seed):
    b = _batch(case, seed)
    table, requests, _ = _tables(b, case["page"], case["max_pages"], case["slots"], seed)
    n, ps = requests.size, case["page"]
    out = {"offsets": np.zeros(n + 1, dtype=np.int32), "lens": np.zeros(n, dtype=np.int32), "tables": np.full((n, case["max_pages"]), -1, dtype=np.int32)}
    for k in ("entries", "positions", "rows"):
        out[k] = np.full(b["max_tokens"], -1, dtype=np.int32)
    at = 0
    for i in range(n):
        if requests[i] >= 0:
            pos = np.arange(b["old"][i], b["new"][i])
            end = at + pos.size
            out["entries"][at:end], out["positions"][at:end] = i, pos
            out["rows"][at:end] = table[requests[i], pos // ps] * ps + pos % ps
            out["lens"][i] = b["new"][i]
            held = -(-int(b["new"][i]) // ps)
            out["tables"][i, :held] = table[requests[i], :held]
            at = end
        out["offsets"][i + 1] = at
    return {k: out[k] for k in ("offsets", "lens", "entries", "positions", "rows", "tables")}


def _decode64(rec):
    """Rows' bytes to 64-bit values [n, 576], from the formats' definitions."""
    c = rec[:, :LATENT].long()
    e, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e == 0, m / 512.0, (1.0 + m / 8.0) * torch.pow(2.0, (e - 7).double()))
    scale = rec[:, LATENT:LATENT + 16].contiguous().view(torch.float32).double()
    lat = torch.where(c >= 128, -mag, mag) * scale.repeat_interleave(BLOCK, 1)
    w = rec[:, LATENT + 16:].contiguous().view(torch.int16).int() << 16
    return torch.cat((lat, w.view(torch.float32).double()), 1)


def _exact_rows(case, seed):
    st = prepare(case, seed)
    kv = st["kv"].double().cpu().numpy()
    lat = kv[:, :LATENT]
    norm = np.sqrt(np.square(lat).sum(1) / LATENT + np.float64(np.float32(EPS)))
    y = (lat * st["weight"].double().cpu().numpy()) / norm[:, None]
    for b in range(0, LATENT, BLOCK):
        blk = y[:, b:b + BLOCK]
        top = np.abs(blk).max(1)
        k = np.ceil(np.log2(top / 448.0))
        k = np.where(top > 448.0 * 2.0 ** k, k + 1, np.where(top <= 448.0 * 2.0 ** (k - 1), k - 1, k))
        s = 2.0 ** k[:, None]
        a = np.abs(blk) / s
        step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -12))), -6) - 3)
        blk[...] = np.copysign(np.rint(a / step) * step * s, blk)
    cs = st["rope"][st["positions"].long()].double().cpu().numpy()
    z = (kv[:, LATENT::2] + 1j * kv[:, LATENT + 1::2]) * (cs[:, :ROPE // 2] + 1j * cs[:, ROPE // 2:])
    turned = np.stack((z.real, z.imag), -1).reshape(-1, ROPE)
    values = _decode64(st["pool"])
    rows = st["rows"].long()
    ok = rows >= 0
    values[rows[ok]] = torch.from_numpy(np.concatenate((y, turned), 1)).cuda()[ok]
    back = st["back"].long()
    out = values[back.clamp(min=0)]
    out[back < 0] = 0.0
    return out


def _exact_chunk(case, seed):
    if work(case)["flops"] > 6e12:
        return None
    st = prepare(case, seed)
    h, ps = case["heads"], case["page"]
    o = torch.zeros(st["o"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["lse"].shape, dtype=torch.float64, device="cuda")
    for i in range(st["lens_host"].size):
        first, count, length = int(st["offsets_host"][i]), int(st["offsets_host"][i + 1] - st["offsets_host"][i]), int(st["lens_host"][i])
        if count == 0:
            continue
        pages = st["tables"][i, :-(-length // ps)].long()
        rows = (pages[:, None] * ps + torch.arange(ps, device="cuda")).flatten()[:length]
        kv = _decode64(st["pool"][rows])
        # in runs of queries, each over the rows up to its last query's
        per = max(1, min(count, int(1e8) // (h * length)))
        for j in range(0, count, per):
            m = min(per, count - j)
            end = length - count + j + m
            s = (st["q"][first + j:first + j + m].double().reshape(m * h, DIMS) @ kv[:end].T) * SM_SCALE
            seen = torch.ones(m, end, dtype=torch.bool, device="cuda").tril(end - m)
            s = s.view(m, h, end).masked_fill(~seen[:, None], -math.inf)
            l = torch.logsumexp(s, -1)
            lse[first + j:first + j + m] = l
            o[first + j:first + j + m] = (torch.exp(s - l[..., None]).view(m * h, end) @ kv[:end, :LATENT]).view(m, h, LATENT)
    return o, lse


def exact(case, seed):
    return {"plan": _exact_plan, "rows": _exact_rows, "chunk": _exact_chunk}[case["kind"]](case, seed)
