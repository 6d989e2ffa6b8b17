"""Cases of the 4-bit MLA cache's operators, their plain forms, and what they have to compute.

The operators work on rows of a paged device pool that hold one token's MLA key/value in 4 bits:
416 bytes = 256 B of e2m1 codes (512 latent dims, even dim in the low nibble), 32 B of e4m3 scales
(one per 16 dims) and 128 B of bf16 RoPE values (64 dims). A latent value is
code x scale x latent_scale, latent_scale a power of two of the caller's.

kind "rows":    hs_fp4_pack_rows writes new tokens' rows, hs_fp4_unpack_rows reads rows back as bf16
kind "sparse":  hs_fp4_sparse_mla_decode, attention over the rows of a row table
kind "window":  hs_fp4_window_mla_decode, attention over the last `window` tokens and the first
                `sinks` tokens of each sequence, through its page table, for one or more new tokens
kind "fork":    hs_pages_extend + hs_pages_fork, a step in which sequences grow and branch
kind "compact": hs_pages_free + hs_pages_compact, finished sequences leave and the pool is packed
"""
import math

import numpy as np
import torch

own = False

ROW, LATENT, ROPE, DIMS, BLOCK = 416, 512, 64, 576, 16
SM_SCALE = 1.0 / math.sqrt(192.0)
HALF_STEPS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)  # between the e2m1 magnitudes 0 .5 1 1.5 2 3 4 6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def listed():
    return [
        # one decode step of the 32-request DSA workload writes its tokens' rows and reads them back
        {"name": "rows_step", "kind": "rows", "n": 32, "m": 32, "pool_rows": 4096, "stride": 576, "latent_scale": 1.0},
        # a prefill chunk is written, and twice as many rows are staged for its attention
        {"name": "rows_prefill", "kind": "rows", "n": 32768, "m": 65536, "pool_rows": 131072, "stride": 640, "latent_scale": 0.25},
        # the tiny workload: two requests, top 64, the 16 heads of one tensor-parallel rank
        {"name": "sparse_tiny", "kind": "sparse", "requests": 2, "heads": 16, "top_k": 64, "pool_rows": 256, "masked": 0.0},
        # the DSA decode step: 32 requests, 128 heads, top 2,048
        {"name": "sparse_dsa", "kind": "sparse", "requests": 32, "heads": 128, "top_k": 2048, "pool_rows": 69632, "masked": 0.02},
        # the IndexShare step's 256 requests, one layer
        {"name": "sparse_256", "kind": "sparse", "requests": 256, "heads": 128, "top_k": 2048, "pool_rows": 540672, "masked": 0.02},
        # one short chat request on one of eight ranks: latency
        {"name": "window_one", "kind": "window", "requests": 1, "heads": 16, "queries": 1, "window": 127, "sinks": 3,
         "lo": 700, "hi": 1000, "page": 64, "pad": 0},
        # verify steps of a speculative batch (three drafts and the sampled token), 16 heads
        {"name": "window_verify", "kind": "window", "requests": 32, "heads": 16, "queries": 4, "window": 1024, "sinks": 4,
         "lo": 500, "hi": 32768, "page": 64, "pad": 2},
        # a large batch with every head over a long window
        {"name": "window_long", "kind": "window", "requests": 64, "heads": 128, "queries": 1, "window": 8192, "sinks": 64,
         "lo": 4096, "hi": 32768, "page": 64, "pad": 0},
        # best-of-2 of four sequences
        {"name": "fork_few", "kind": "fork", "slots": 16, "parents": 4, "children": 1, "grow": 1, "lo": 200, "hi": 4000,
         "max_pages": 128, "page": 64, "layers": 1, "spare": 16},
        # 64 beams: every sequence takes 100 tokens (an accepted prompt turn), then three children each, four layers
        {"name": "fork_beams", "kind": "fork", "slots": 256, "parents": 64, "children": 3, "grow": 100, "lo": 2000, "hi": 12000,
         "max_pages": 512, "page": 64, "layers": 4, "spare": 512},
        # a few finished sequences of a small pool
        {"name": "compact_few", "kind": "compact", "slots": 16, "leave": 5, "lo": 100, "hi": 2000, "max_pages": 64, "page": 64,
         "layers": 1, "spare": 40},
        # a third of 128 sequences leave a pool of four layers
        {"name": "compact_pool", "kind": "compact", "slots": 128, "leave": 43, "lo": 500, "hi": 6000, "max_pages": 256, "page": 64,
         "layers": 4, "spare": 700},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["rows", "sparse", "sparse", "window", "window", "fork", "compact"])
    if kind == "rows":
        n = _log(rng, 1, 32768)
        m = _log(rng, 1, 65536)
        return {"kind": kind, "n": n, "m": m, "pool_rows": max(n, m) + _log(rng, 1, 50000), "stride": 576 + 8 * rng.choice([0, 0, 1, 8, 64]),
                "latent_scale": 2.0 ** rng.randint(-6, 6)}
    if kind == "sparse":
        heads, k = _log(rng, 1, 128), _log(rng, 1, 4096)
        r = _log(rng, 1, max(1, min(256, 256 * 2048 // k)))
        return {"kind": kind, "requests": r, "heads": heads, "top_k": k, "pool_rows": k + _log(rng, 1, r * k), "masked": rng.choice([0.0, 0.02, 0.5])}
    if kind == "window":
        window, sinks, heads = _log(rng, 1, 8192), rng.choice([0, 1, 4, _log(rng, 1, 64)]), _log(rng, 1, 128)
        queries = rng.choice([1, 1, 1, 2, 3, 4, 8])
        r = max(1, _log(rng, 1, 64) // (queries if heads * queries > 128 else 1))
        hi = _log(rng, 16, 32768)
        return {"kind": kind, "requests": r, "heads": heads, "queries": queries, "window": window, "sinks": sinks, "lo": _log(rng, 1, hi), "hi": hi,
                "page": rng.choice([1, 16, 48, 64, 128]), "pad": rng.randint(0, r // 4)}
    layers = rng.choice([1, 2, 4])
    page = rng.choice([16, 64, 64, 128])
    if kind == "fork":
        parents, children = _log(rng, 1, 64), rng.choice([1, 2, 3])
        lo = _log(rng, 1, 4000)
        return {"kind": kind, "slots": parents * (children + 1) + rng.randint(0, 9), "parents": parents, "children": children, "grow": _log(rng, 1, 500),
                "lo": lo, "hi": lo + _log(rng, 1, 4000), "max_pages": 9000 // page + rng.randint(0, 40), "page": page, "layers": layers, "spare": _log(rng, 1, 2000)}
    slots = _log(rng, 1, 128)
    lo = _log(rng, 1, 3000)
    return {"kind": kind, "slots": slots, "leave": rng.randint(0, slots), "lo": lo, "hi": lo + _log(rng, 1, 2800), "max_pages": 5900 // page + rng.randint(0, 40),
            "page": page, "layers": layers, "spare": _log(rng, 1, 700)}


def work(case):
    """Each input read once and each output written once; the two matrix products of attention."""
    k = case["kind"]
    if k == "rows":
        return {"bytes": case["n"] * (DIMS * 2 + 4 + ROW) + case["m"] * (ROW + 4 + DIMS * 2), "flops": 0}
    if k == "sparse":
        r, h, n = case["requests"], case["heads"], case["top_k"]
        live = r * n * (1 - case["masked"])
        rows = min(live, case["pool_rows"])
        return {"bytes": rows * ROW + r * n * 4 + r * h * (DIMS * 2 + LATENT * 2 + 4), "flops": 2 * live * h * (DIMS + LATENT)}
    if k == "window":
        s = np.asarray(_lengths(case, 0), dtype=np.float64)
        h, q, w, sink = case["heads"], case["queries"], case["window"], case["sinks"]
        seen = sum(float((np.minimum(np.maximum(s - q + i + 1, 0), w + sink)).sum()) for i in range(q))
        rows = float(np.minimum(s, w + sink + q - 1).sum())
        n = case["requests"] * q * h
        return {"bytes": rows * (ROW + 4 / case["page"]) + n * (DIMS * 2 + LATENT * 2 + 4), "flops": 2 * seen * h * (DIMS + LATENT)}
    s = _pages(case, 0)
    moved = s["moved"] * case["layers"] * ROW
    return {"bytes": 2 * moved + s["ints"], "flops": 0}


# ---------------------------------------------------------------- inputs


def _lengths(case, seed):
    g = np.random.default_rng([seed, 11])
    s = g.integers(case["lo"], case["hi"] + 1, size=case["requests"])
    if case["pad"]:
        s[-case["pad"]:] = 0  # a padded batch: the last requests are empty
    return s.astype(np.int64)


def _new_rows(gen, n):
    """bf16 latents (normed: unit spread, a few loud dims) and RoPE values of n tokens, on the GPU."""
    gain = torch.ones(DIMS, device="cuda")
    gain[:LATENT:37] = 6.0
    gain[5:LATENT:11] = 0.05
    return (torch.randn(n, DIMS, generator=gen, device="cuda") * gain).to(torch.bfloat16)


def _pool(gen, rows, latent_scale):
    pool = torch.empty(rows, ROW, dtype=torch.uint8, device="cuda")
    for at in range(0, rows, 65536):
        pool[at:at + 65536] = _quantise(_new_rows(gen, min(65536, rows - at)), latent_scale)
    return pool


def _pages(case, seed):
    """The page tables of a fork or compact case, on the host, and what the pass has to move."""
    g = np.random.default_rng([seed, 12])
    slots, ps, mp, kind = case["slots"], case["page"], case["max_pages"], case["kind"]
    table = np.full((slots, mp), -1, dtype=np.int32)
    busy = case["parents"] if kind == "fork" else slots
    lens = np.zeros(slots, dtype=np.int64)
    # evenly spread page counts, so that the pool has the same size for every seed; the last pages' fill is random
    most = mp * ps - (case["grow"] if kind == "fork" else 0)
    pages_of = -(-np.linspace(case["lo"], min(case["hi"], most), busy).astype(np.int64) // ps)
    lens[:busy] = np.minimum((pages_of - 1) * ps + g.integers(1, ps + 1, size=busy), most)
    lens = lens[g.permutation(slots)]
    held = -(-lens // ps)
    total = int(held.sum())
    pages = total + case["spare"]
    perm = g.permutation(pages).astype(np.int32)
    at = 0
    for r in range(slots):
        table[r, :held[r]] = perm[at:at + held[r]]
        at += held[r]
    refs = np.zeros(pages, dtype=np.int32)
    refs[perm[:total]] = 1
    if kind == "compact":  # half of the sequences share their first page with the sequence before them
        for r in range(1, slots, 2):
            old, new = table[r, 0], table[r - 1, 0]
            if old >= 0 and new >= 0 and refs[old] == 1:
                refs[old], refs[new], table[r, 0] = 0, refs[new] + 1, new
    free = np.zeros(pages, dtype=np.int32)
    spare = np.flatnonzero(refs == 0).astype(np.int32)
    spare = spare[g.permutation(spare.size)]
    free[:spare.size] = spare
    s = {"table": table, "refs": refs, "free": free, "count": np.array([spare.size], dtype=np.int32), "pages": pages, "lens": lens}
    active = np.flatnonzero(lens > 0)
    if kind == "fork":
        s["grown"] = active.astype(np.int32)
        s["old"] = lens[active].astype(np.int32)
        s["new"] = (lens[active] + case["grow"]).astype(np.int32)
        idle = np.flatnonzero(lens == 0)[: active.size * case["children"]]
        s["parents"] = np.repeat(active, case["children"])[: idle.size].astype(np.int32)
        s["children"] = idle.astype(np.int32)
        s["fork_lens"] = (np.repeat(lens[active], case["children"])[: idle.size] + case["grow"]).astype(np.int32)
        s["moved"] = int((s["fork_lens"] % ps).sum())
        s["ints"] = 4 * int((2 * -(-s["fork_lens"] // ps)).sum() + 8 * idle.size)
    else:
        s["leave"] = np.sort(g.permutation(slots)[: case["leave"]]).astype(np.int32)
        drop = np.bincount(table[s["leave"]][table[s["leave"]] >= 0], minlength=pages)
        alive = (refs - drop) > 0
        s["moved"] = int(alive[int(alive.sum()):].sum()) * ps
        s["ints"] = 4 * (2 * slots * mp + 3 * pages)
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)
    k = case["kind"]
    st = {"case": dict(case), "keep": {}}
    if k == "rows":
        g, n, m, total = case["latent_scale"], case["n"], case["m"], case["pool_rows"]
        st["scale"] = g
        wide = torch.randn(n, case["stride"], generator=gen, device="cuda").to(torch.bfloat16)
        wide[:, :DIMS] = _new_rows(gen, n) * g
        st["kv"] = wide[:, :DIMS]  # a slice of a wider projection
        order = torch.randperm(total, generator=gen, device="cuda")
        rows = order[:n].to(torch.int32)
        rows[torch.rand(n, generator=gen, device="cuda") < 0.02] = -1  # padding tokens of the batch
        st["rows"] = rows
        st["pool"] = _pool(gen, total, g)
        back = order[torch.randperm(max(n, m), generator=gen, device="cuda")[:m]].to(torch.int32)
        back[torch.rand(m, generator=gen, device="cuda") < 0.02] = -1
        st["back"] = back
        return st
    if k == "sparse":
        r, n = case["requests"], case["top_k"]
        st["scale"] = 1.0
        st["q"] = torch.randn(r, case["heads"], DIMS, generator=gen, device="cuda").to(torch.bfloat16)
        st["pool"] = _pool(gen, case["pool_rows"], 1.0)
        # a resolved step: distinct rows for every entry as far as the pool has them
        lots = torch.cat([torch.randperm(case["pool_rows"], generator=gen, device="cuda") for _ in range(-(-r * n // case["pool_rows"]))])
        rows = lots[: r * n].reshape(r, n).to(torch.int32)
        rows[torch.rand(r, n, generator=gen, device="cuda") < case["masked"]] = -1
        st["rows"] = rows.contiguous()
        return st
    if k == "window":
        r, ps, w, sink, nq = case["requests"], case["page"], case["window"], case["sinks"], case["queries"]
        s = _lengths(case, seed)
        mp = int(max(1, -(-case["hi"] // ps)))
        # pages that some query of the step sees are on the GPU; those between are not
        first = np.maximum(s - nq - w + 1, 0) // ps
        held = -(-s // ps)
        idx = np.arange(mp)[None]
        need = (idx < held[:, None]) & ((idx >= first[:, None]) | (idx * ps < sink))
        table = np.full((r, mp), -1, dtype=np.int32)
        total = int(need.sum())
        table[need] = np.random.default_rng([seed, 13]).permutation(total).astype(np.int32)
        st["scale"] = 0.5
        st["pool"] = _pool(gen, max(1, total) * ps, 0.5)
        st["table"] = torch.from_numpy(table).cuda()
        st["lens"] = torch.from_numpy(s.astype(np.int32)).cuda()
        st["q"] = torch.randn(r, nq, case["heads"], DIMS, generator=gen, device="cuda").to(torch.bfloat16)
        return st
    h = _pages(case, seed)
    st["pages"] = h["pages"]
    st["pools"] = [torch.randint(0, 256, (h["pages"] * case["page"], ROW), generator=gen, device="cuda", dtype=torch.uint8) for _ in range(case["layers"])]
    # the integer state in one buffer, and as it stands before the pass
    flat = np.concatenate([h["table"].reshape(-1), h["refs"], h["free"], h["count"]])
    st["before"] = torch.from_numpy(flat).cuda()
    st["ints"] = st["before"].clone()
    a, b, c = h["table"].size, h["table"].size + h["pages"], h["table"].size + 2 * h["pages"]
    st["table"], st["refs"] = st["ints"][:a].view(case["slots"], case["max_pages"]), st["ints"][a:b]
    st["free"], st["count"] = st["ints"][b:c], st["ints"][c:]
    for name in ("grown", "old", "new", "parents", "children", "fork_lens", "leave"):
        if name in h:
            st[name] = torch.from_numpy(h[name]).cuda()
    return st


# ---------------------------------------------------------------- plain forms


def _quantise(kv, latent_scale):
    """Rows' bytes of bf16 tokens [n, 576]: e4m3(amax / 6) per 16 dims, then the nearest e2m1 value."""
    n = kv.shape[0]
    x = (kv[:, :LATENT].float() / latent_scale).view(n, LATENT // BLOCK, BLOCK)
    scale = (x.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.float()[..., None]
    a = torch.where(s > 0, x.abs() / s, torch.zeros_like(x))
    code = torch.zeros_like(x, dtype=torch.uint8)
    for i, half in enumerate(HALF_STEPS):  # a value halfway goes to the even code
        code += (a > half) if i % 2 == 0 else (a >= half)
    code |= (x < 0).to(torch.uint8) << 3
    code = code.view(n, LATENT)
    out = torch.empty(n, ROW, dtype=torch.uint8, device=kv.device)
    out[:, :256] = code[:, 0::2] | (code[:, 1::2] << 4)
    out[:, 256:288] = scale.view(torch.uint8)
    out[:, 288:] = kv[:, LATENT:].contiguous().view(torch.uint8)
    return out


def _values(rec, latent_scale):
    """(latent [..., 512], rope [..., 64]) in 32 bits of rows' bytes [..., 416]."""
    lut = torch.tensor(E2M1, device=rec.device)
    codes = rec[..., :256].int()
    lat = torch.stack((lut[codes & 15], lut[codes >> 4]), dim=-1).reshape(*rec.shape[:-1], LATENT // BLOCK, BLOCK)
    scale = rec[..., 256:288].contiguous().view(torch.float8_e4m3fn).float() * latent_scale
    rope = rec[..., 288:].contiguous().view(torch.bfloat16).float()
    return (lat * scale[..., None]).reshape(*rec.shape[:-1], LATENT), rope


def _attend(q, lat, rope, seen):
    """q [R, M, 576], lat [R, T, 512], rope [R, T, 64], seen [R, M or 1, T] -> o bf16, lse."""
    q = q.float()
    s = (torch.matmul(q[..., :LATENT], lat.transpose(1, 2)) + torch.matmul(q[..., LATENT:], rope.transpose(1, 2))) * SM_SCALE
    s = torch.where(seen, s, torch.full((), -math.inf, device=s.device))
    top = s.amax(-1, keepdim=True)
    safe = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(s - safe)
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p, lat) / torch.where(z > 0, z, torch.ones_like(z))
    return o.to(torch.bfloat16), (top + torch.log(torch.where(z > 0, z, torch.ones_like(z))))[..., 0]


def _plain_rows(st):
    rows, back, total = st["rows"], st["back"], st["pool"].shape[0]
    ok = rows >= 0
    st["pool"][rows[ok].long()] = _quantise(st["kv"], st["scale"])[ok]
    live = (back >= 0) & (back < total)
    lat, rope = _values(st["pool"][back.clamp(min=0).long()], st["scale"])
    return torch.where(live[:, None], torch.cat((lat, rope), -1), torch.zeros((), device=rows.device)).to(torch.bfloat16)


def _plain_sparse(st):
    lat, rope = _values(st["pool"][st["rows"].clamp(min=0).long()], st["scale"])
    return _attend(st["q"], lat, rope, (st["rows"] >= 0)[:, None, :])


def _plain_window(st):
    c, q, lens = st["case"], st["q"], st["lens"].long()
    r, nq, h, _ = q.shape
    w, sinks, ps = c["window"], c["sinks"], c["page"]
    kept = lens.clamp(max=sinks)  # tokens 0 .. kept - 1, then from `start` to the end
    start = torch.maximum(kept, lens.sub(nq).clamp(min=0) - w + 1)
    j = torch.arange(min(sinks + w + nq - 1, c["hi"]), device=q.device)[None]
    t = torch.where(j < kept[:, None], j, start[:, None] + j - kept[:, None])
    there = t < lens[:, None]
    safe = torch.where(there, t, torch.zeros_like(t))
    page = st["table"].long().gather(1, safe // ps)
    lat, rope = _values(st["pool"][(page * ps + safe % ps).clamp(min=0)], st["scale"])
    at = lens[:, None] - nq + torch.arange(nq, device=q.device)[None]  # [R, Q] positions of the queries
    seen = (there & (page >= 0))[:, None] & (t[:, None] <= at[..., None]) & ((t[:, None] < sinks) | (t[:, None] > at[..., None] - w))
    o, lse = _attend(q.reshape(r, nq * h, DIMS), lat, rope, seen.repeat_interleave(h, dim=1))
    return o.view(r, nq, h, LATENT), lse.view(r, nq, h)


def _take(st, need):
    """How many pages each entry gets (-1: none are left for it) and where its first stands from the stack's top."""
    cum = torch.cumsum(need, 0)
    given = torch.where((need > 0) & (cum > st["count"]), torch.full_like(need, -1), need)
    return given, cum - need


def _plain_fork(st):
    c, ps, dev = st["case"], st["case"]["page"], st["ints"].device
    st["ints"].copy_(st["before"])
    table, refs, free, count = st["table"], st["refs"], st["free"], st["count"]
    # sequences grow: pages for the tokens past the ones that they hold
    a, b = (st["old"].long() + ps - 1) // ps, (st["new"].long() + ps - 1) // ps
    given, first = _take(st, b - a)
    k = torch.arange(c["grow"] // ps + 1, device=dev)[None]
    m = k < given[:, None]
    new = free[(count - 1 - first[:, None] - k).clamp(min=0).long()]
    table[st["grown"].long()[:, None].expand_as(m)[m], (a[:, None] + k)[m]] = new[m]
    refs[new[m].long()] = 1
    count -= given.clamp(min=0).sum().int()
    grown = given.int()
    # they branch: whole pages are shared, a page that is not full is copied
    lens, par, chi = st["fork_lens"].long(), st["parents"].long(), st["children"].long()
    idx = torch.arange(c["max_pages"], device=dev)[None]
    src = table[par]
    part = src.gather(1, (lens // ps).clamp(max=c["max_pages"] - 1)[:, None])[:, 0]
    part = torch.where(lens % ps > 0, part, torch.full_like(part, -1))
    given, first = _take(st, (part >= 0).long())
    ok = given >= 0
    whole = (idx < (lens // ps)[:, None]) & (src >= 0) & ok[:, None]
    table[chi] = torch.where(whole, src, torch.full_like(src, -1))
    refs.index_add_(0, src[whole].long(), torch.ones((), dtype=torch.int32, device=dev).expand(int(whole.sum())))
    took = given > 0
    new = free[(count - 1 - first).clamp(min=0).long()][took]
    table[chi[took], (lens // ps)[took]] = new
    refs[new.long()] = 1
    count -= given.clamp(min=0).sum().int()
    j = torch.arange(ps, device=dev)[None]
    live = j < (lens % ps)[took][:, None]
    old, to = (part[took].long()[:, None] * ps + j)[live], (new.long()[:, None] * ps + j)[live]
    for pool in st["pools"]:
        pool[to] = pool[old]
    return {"ints": st["ints"], "pools": st["pools"], "grown": grown, "forked": given.int()}


def _plain_compact(st):
    c, ps, dev = st["case"], st["case"]["page"], st["ints"].device
    st["ints"].copy_(st["before"])
    table, refs, free, count = st["table"], st["refs"], st["free"], st["count"]
    # the leaving sequences' entries go; pages that nobody holds go onto the stack, the lowest on top
    gone = table[st["leave"].long()]
    drop = gone[gone >= 0].long()
    refs.index_add_(0, drop, torch.full_like(drop, -1, dtype=torch.int32))
    table[st["leave"].long()] = -1
    new = torch.unique(drop)
    new = new[refs[new] == 0].flip(0).int()
    free[count.long() + torch.arange(new.numel(), device=dev)] = new
    count += new.numel()
    # the k-th live page past the first `live` pages moves into the k-th free page among them
    n = refs.numel()
    live = int((refs > 0).sum())
    holes = torch.nonzero(refs[:live] == 0)[:, 0]
    movers = torch.nonzero(refs[live:] > 0)[:, 0] + live
    to = torch.arange(n, device=dev)
    to[movers] = holes
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].int(), table))
    refs[holes] = refs[movers]
    refs[live:] = 0
    free[:n - live] = torch.arange(n - 1, live - 1, -1, device=dev, dtype=torch.int32)
    count.fill_(n - live)
    j = torch.arange(ps, device=dev)[None]
    old, new = (movers[:, None] * ps + j).view(-1), (holes[:, None] * ps + j).view(-1)
    for pool in st["pools"]:
        pool[new] = pool[old]
    return {"ints": st["ints"], "pools": st["pools"]}


# ---------------------------------------------------------------- the framework's calls


def _flags(keep):
    if "err" not in keep:
        keep["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return keep["err"]


def _own_rows(st, hs):
    kv, pool, keep = st["kv"], st["pool"], st["keep"]
    out = torch.empty(st["back"].shape[0], DIMS, dtype=torch.bfloat16, device="cuda")
    hs.hs_fp4_pack_rows(kv.shape[0], kv, kv.stride(0), st["rows"], st["scale"], pool, pool.shape[0], _flags(keep))
    hs.hs_fp4_unpack_rows(out.shape[0], pool, pool.shape[0], st["back"], st["scale"], out, DIMS, _flags(keep))
    return out


def _mla_buffers(st, hs, requests, heads, queries, rows):
    keep = st["keep"]
    if "splits" not in keep:
        keep["splits"] = hs.hs_fp4_mla_splits(requests, heads, queries, rows)
        keep["bytes"] = hs.hs_fp4_mla_workspace_bytes(requests, heads, queries, keep["splits"])
        keep["ws"] = torch.zeros(max(16, keep["bytes"]), dtype=torch.uint8, device="cuda")
    return keep["splits"], keep["ws"], keep["bytes"]


def _own_sparse(st, hs):
    q, pool = st["q"], st["pool"]
    r, h, _ = q.shape
    n = st["rows"].shape[1]
    splits, ws, wsb = _mla_buffers(st, hs, r, h, 1, n)
    o = torch.empty(r, h, LATENT, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(r, h, dtype=torch.float32, device="cuda")
    hs.hs_fp4_sparse_mla_decode(r, h, n, splits, q, pool, pool.shape[0], st["rows"], SM_SCALE, st["scale"], o, lse, ws, wsb, _flags(st["keep"]))
    return o, lse


def _own_window(st, hs):
    c, q, pool = st["case"], st["q"], st["pool"]
    r, nq, h, _ = q.shape
    splits, ws, wsb = _mla_buffers(st, hs, r, h, nq, c["window"] + c["sinks"] + nq - 1)
    o = torch.empty(r, nq, h, LATENT, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(r, nq, h, dtype=torch.float32, device="cuda")
    hs.hs_fp4_window_mla_decode(r, h, nq, c["window"], c["sinks"], splits, q, pool, pool.shape[0], c["page"], st["table"].shape[1], st["lens"], st["table"],
                                SM_SCALE, st["scale"], o, lse, ws, wsb, _flags(st["keep"]))
    return o, lse


def _page_pool(st, hs):
    c, keep = st["case"], st["keep"]
    if "pool" not in keep:
        wsb = hs.hs_pages_workspace_bytes(c["slots"], st["pages"])
        keep["ws"] = torch.zeros(wsb, dtype=torch.uint8, device="cuda")
        keep["pool"] = hs.make_page_pool(st["pools"], c["slots"], c["max_pages"], st["pages"], c["page"], ROW, st["table"], st["refs"], st["free"], st["count"],
                                         keep["ws"], wsb, _flags(keep))
    return keep["pool"]


def _own_fork(st, hs):
    pool = _page_pool(st, hs)
    st["ints"].copy_(st["before"])
    grown = torch.empty_like(st["grown"])
    forked = torch.empty_like(st["children"])
    hs.hs_pages_extend(pool, grown.numel(), st["grown"], st["old"], st["new"], grown)
    hs.hs_pages_fork(pool, forked.numel(), st["parents"], st["children"], st["fork_lens"], forked)
    return {"ints": st["ints"], "pools": st["pools"], "grown": grown, "forked": forked}


def _own_compact(st, hs):
    pool = _page_pool(st, hs)
    st["ints"].copy_(st["before"])
    hs.hs_pages_free(pool, st["leave"].numel(), st["leave"])
    hs.hs_pages_compact(pool)
    return {"ints": st["ints"], "pools": st["pools"]}


def run(state):
    kind = state["case"]["kind"]
    if own:
        import hierarchical_sparse_attention_gb300 as hs

        return {"rows": _own_rows, "sparse": _own_sparse, "window": _own_window, "fork": _own_fork, "compact": _own_compact}[kind](state, hs)
    return {"rows": _plain_rows, "sparse": _plain_sparse, "window": _plain_window, "fork": _plain_fork, "compact": _plain_compact}[kind](state)


# ---------------------------------------------------------------- the definitions in 64 bits, on the host


def _e4m3(code):
    e, m = code >> 3, code & 7
    return m / 8.0 * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)


def _nearest(x, values):
    """Index of the nearest of ascending `values` (halfway: the even index; past the end: the last)."""
    mid = (values[1:] + values[:-1]) / 2
    lo, hi = np.searchsorted(mid, x, side="left"), np.searchsorted(mid, x, side="right")
    return np.where((hi > lo) & (lo % 2 == 1), hi, lo)


def _decode64(rec, g):
    code = np.empty((rec.shape[0], LATENT), dtype=np.uint8)
    code[:, 0::2], code[:, 1::2] = rec[:, :256] & 15, rec[:, :256] >> 4
    mags = np.array(E2M1, dtype=np.float64)
    by = np.array([_e4m3(i) for i in range(127)] + [np.nan])
    scale = by[rec[:, 256:288] & 127] * np.where(rec[:, 256:288] & 128, -1.0, 1.0)
    rope = (np.ascontiguousarray(rec[:, 288:]).view("<u2").astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    return mags[code] * np.repeat(scale, BLOCK, axis=1) * g, rope


def _softmax64(q, lat, rope):
    """One request's heads over the rows that it sees."""
    if lat.shape[0] == 0:
        return np.zeros((q.shape[0], LATENT)), np.full(q.shape[0], -np.inf)
    s = (q @ np.concatenate((lat, rope), axis=1).T) * SM_SCALE
    top = s.max(axis=1, keepdims=True)
    e = np.exp(s - top)
    z = e.sum(axis=1, keepdims=True)
    return (e @ lat) / z, (top + np.log(z))[:, 0]


def _exact_pages(case, st):
    ints = st["before"].cpu().numpy().copy()
    pools = [p.cpu().numpy().copy() for p in st["pools"]]
    ps, mp, n = case["page"], case["max_pages"], st["pages"]
    a = case["slots"] * mp
    table, refs, free, count = ints[:a].reshape(-1, mp), ints[a:a + n], ints[a + n:a + 2 * n], ints[a + 2 * n:]
    host = {k: st[k].cpu().numpy() for k in ("grown", "old", "new", "parents", "children", "fork_lens", "leave") if k in st}

    def grant(needs):
        got, total = [], 0
        for w in needs:
            total += w
            got.append(-1 if w > 0 and total > count[0] else w)
        return got

    def pop():
        count[0] -= 1
        refs[free[count[0]]] = 1
        return free[count[0]]

    out = {"ints": ints, "pools": pools}
    if case["kind"] == "fork":
        ceil = lambda x: -(-int(x) // ps)  # noqa: E731
        got = grant([ceil(w) - ceil(o) for o, w in zip(host["old"], host["new"])])
        for r, o, w in zip(host["grown"], host["old"], got):
            for i in range(max(0, w)):
                table[r, ceil(o) + i] = pop()
        out["grown"] = np.array(got, dtype=np.int32)
        parts = [int(table[p, s // ps]) if s % ps else -1 for p, s in zip(host["parents"], host["fork_lens"])]
        got = grant([int(p >= 0) for p in parts])
        for p, ch, s, part, w in zip(host["parents"], host["children"], host["fork_lens"], parts, got):
            if w < 0:
                continue
            whole = table[p, :s // ps]
            table[ch, :s // ps] = whole
            np.add.at(refs, whole[whole >= 0], 1)
            if w:
                table[ch, s // ps] = pop()
                to = int(table[ch, s // ps])
                for x in pools:
                    x[to * ps:to * ps + s % ps] = x[part * ps:part * ps + s % ps]
        out["forked"] = np.array(got, dtype=np.int32)
        return out
    gone = set()
    for r in host["leave"]:
        for p in table[r][table[r] >= 0]:
            refs[p] -= 1
            if refs[p] == 0:
                gone.add(int(p))
        table[r] = -1
    for p in sorted(gone, reverse=True):
        free[count[0]] = p
        count[0] += 1
    live = int((refs > 0).sum())
    pairs = list(zip([p for p in range(live, n) if refs[p] > 0], [p for p in range(live) if refs[p] == 0]))
    to = np.arange(n, dtype=np.int32)
    for p, h in pairs:
        to[p], refs[h], refs[p] = h, refs[p], 0
        for x in pools:
            x[h * ps:(h + 1) * ps] = x[p * ps:(p + 1) * ps]
    table[table >= 0] = to[table[table >= 0]]
    free[:n - live] = np.arange(n - 1, live - 1, -1)
    count[0] = n - live
    return out


def exact(case, seed):
    st = prepare(case, seed)
    k = case["kind"]
    if k in ("fork", "compact"):
        return _exact_pages(case, st)
    pool, g = st["pool"].cpu().numpy(), float(st["scale"])
    if k == "rows":
        kv, rows, back = st["kv"].double().cpu().numpy(), st["rows"].cpu().numpy(), st["back"].cpu().numpy()
        lat, rope = _decode64(pool[np.maximum(back, 0)], g)
        value = np.concatenate((lat, rope), axis=1)
        value[back < 0] = 0
        x = (kv[:, :LATENT] / g).reshape(len(rows), -1, BLOCK)
        steps, mags = np.array([_e4m3(i) for i in range(127)]), np.array(E2M1[:8])
        s = steps[_nearest(np.abs(x).max(-1) / 6.0, steps)][..., None]
        new = np.where(s > 0, mags[_nearest(np.abs(x) / np.where(s > 0, s, 1.0), mags)] * np.sign(x) * s * g, 0.0).reshape(len(rows), LATENT)
        new = np.concatenate((new, kv[:, LATENT:]), axis=1)
        where = np.full(pool.shape[0], -1)
        where[rows[rows >= 0]] = np.flatnonzero(rows >= 0)
        at = np.where(back >= 0, where[np.maximum(back, 0)], -1)
        value[at >= 0] = new[at[at >= 0]]
        return value
    q = st["q"].double().cpu().numpy()
    o, lse = np.zeros(q.shape[:-1] + (LATENT,)), np.full(q.shape[:-1], -np.inf)
    if k == "sparse":
        rows = st["rows"].cpu().numpy()
        for r in range(q.shape[0]):
            o[r], lse[r] = _softmax64(q[r], *_decode64(pool[rows[r][rows[r] >= 0]], g))
        return o, lse
    lens, table = st["lens"].cpu().numpy(), st["table"].cpu().numpy()
    ps, nq = case["page"], case["queries"]
    for r in range(q.shape[0]):
        for i in range(nq):
            at = int(lens[r]) - nq + i
            t = np.array([x for x in range(at + 1) if x < case["sinks"] or x > at - case["window"]], dtype=np.int64)
            if t.size:
                page = table[r, t // ps].astype(np.int64)
                o[r, i], lse[r, i] = _softmax64(q[r, i], *_decode64(pool[(page * ps + t % ps)[page >= 0]], g))
    return o, lse
