"""What the calls of a step with several new tokens refuse on the host, and their limits (no GPU)."""
import os
import re

import pytest

A = 1 << 20  # an aligned stand-in address: nothing is launched in these calls
HEADER = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "hs.h")).read()


def _hs():
    import hierarchical_sparse_attention_gb300 as hs
    return hs


def plan(**kw):
    a = dict(n=4, requests=A, old_lens=A, new_lens=A, num_requests=8, resident_pages=A, max_pages=16, page_size=64, pool_rows=4096, max_tokens=32, token_offsets=A,
             seq_lens=A, entries=A, positions=A, rows=A, max_blocks=16, block_tables=A, error_flags=A)
    a.update(kw)
    _hs().hs_batch_plan(**a)


def pack(**kw):
    a = dict(n=4, kv=A, kv_stride=576, rows=A, norm_weight=A, norm_eps=1e-6, positions=A, rope_table=A, rope_positions=100, pool=A, pool_rows=64, error_flags=A)
    a.update(kw)
    _hs().hs_fp8_pack_rows(**a)


def unpack(**kw):
    a = dict(n=4, pool=A, pool_rows=64, rows=A, kv=A, kv_stride=576, error_flags=A)
    a.update(kw)
    _hs().hs_fp8_unpack_rows(**a)


def chunk(**kw):
    a = dict(n=4, num_heads=16, max_tokens=32, token_offsets=A, seq_lens=A, q=A, kv_pool=A, pool_rows=4096, page_size=64, max_blocks=16, block_tables=A, sm_scale=0.1, o=A,
             lse=A, max_kv_tokens=4096, workspace=A, workspace_bytes=1 << 40, error_flags=A)
    a.update(kw)
    _hs().hs_chunk_mla(**a)


CASES = [(plan, k, v) for k, v in [("n", -1), ("n", 65537), ("num_requests", 0), ("num_requests", 65537), ("max_pages", 0), ("page_size", 0), ("page_size", 2 ** 31 - 1),
                                   ("pool_rows", 0), ("pool_rows", 2 ** 31), ("max_tokens", -1), ("max_tokens", 2 ** 20 + 1), ("max_blocks", 0), ("token_offsets", None),
                                   ("error_flags", None), ("requests", None), ("old_lens", None), ("new_lens", None), ("resident_pages", None)]]
CASES += [(pack, k, v) for k, v in [("n", -1), ("kv_stride", 568), ("kv_stride", 580), ("pool_rows", 0), ("kv", None), ("kv", A + 8), ("rows", None), ("pool", None), ("pool", A + 8),
                                    ("error_flags", None), ("norm_weight", A + 8), ("norm_eps", -1e-6), ("norm_eps", float("nan")), ("norm_eps", float("inf")), ("positions", None),
                                    ("rope_table", None), ("rope_positions", 0)]]
CASES += [(unpack, k, v) for k, v in [("n", -1), ("kv_stride", 568), ("kv_stride", 580), ("pool_rows", 0), ("kv", None), ("kv", A + 8), ("rows", None), ("pool", None),
                                      ("error_flags", None)]]
CASES += [(chunk, k, v) for k, v in [("n", -1), ("n", 65537), ("num_heads", 0), ("num_heads", 129), ("max_tokens", -1), ("max_tokens", 2 ** 20 + 1), ("pool_rows", 0),
                                     ("pool_rows", 2 ** 31), ("page_size", 0), ("max_blocks", 0), ("page_size", 2 ** 31 - 1), ("sm_scale", float("nan")), ("sm_scale", float("inf")),
                                     ("sm_scale", 3e38), ("sm_scale", -3e38), ("max_kv_tokens", -64), ("max_kv_tokens", 100), ("max_kv_tokens", 2 ** 31), ("token_offsets", None),
                                     ("seq_lens", None), ("q", None), ("q", A + 8), ("kv_pool", None), ("kv_pool", A + 8), ("block_tables", None), ("o", None), ("o", A + 8),
                                     ("lse", None), ("workspace", None), ("workspace", A + 128), ("workspace_bytes", 16), ("error_flags", None)]]


@pytest.mark.parametrize("call,name,value", CASES, ids=lambda x: getattr(x, "__name__", str(x)))
def test_refused_on_the_host(call, name, value):
    hs = _hs()
    with pytest.raises(hs.HsError) as e:
        call(**{name: value})
    assert e.value.status == hs.HS_ERR_INVALID_ARG


def test_nothing_to_do_needs_no_arrays():
    none = dict.fromkeys(("rows", "norm_weight", "positions", "rope_table", "pool", "error_flags", "kv"))
    pack(n=0, **none)
    unpack(n=0, pool=None, rows=None, kv=None, error_flags=None)
    off = dict.fromkeys(("token_offsets", "seq_lens", "q", "kv_pool", "block_tables", "o", "lse", "workspace", "error_flags"))
    chunk(n=0, workspace_bytes=0, **off)
    chunk(max_tokens=0, workspace_bytes=0, **off)


def test_limits_are_the_header_s():
    hs = _hs()
    for name in ("HS_MAX_BATCH_ENTRIES", "HS_MAX_BATCH_TOKENS", "HS_FP8_ROW_BYTES", "HS_FLAG_FULL"):
        assert eval(re.search(r"#define %s\s+(\(.*?\)|\d+)" % name, HEADER).group(1), {}) == getattr(hs, name)


@pytest.mark.parametrize("heads", [1, 16, 65, 128])
def test_workspace_sizes(heads):
    hs = _hs()
    size = hs.hs_chunk_mla_workspace_bytes
    assert 0 < size(1, heads, 1, 0) <= size(1, heads, 1, 64) <= size(4, heads, 100, 6400)
    assert size(4, heads, 100, 6400) % 256 == 0
    assert size(0, heads, 1, 64) == size(1, 0, 1, 64) == size(1, 129, 1, 64) == size(1, heads, 1, 63) == size(1, heads, 2 ** 20 + 1, 64) == 0
    assert size(65536, heads, 2 ** 20, (2 ** 31 - 64) // 64 * 64) > 0


def test_tensors_that_the_kernels_cannot_read_are_refused():
    torch = pytest.importorskip("torch")
    ints, bf = torch.zeros(32, dtype=torch.int32), torch.zeros(4, 576, dtype=torch.bfloat16)
    for call, names in ((plan, ("requests", "old_lens", "new_lens", "resident_pages", "token_offsets", "seq_lens", "entries", "positions", "rows", "block_tables", "error_flags")),
                        (pack, ("rows", "positions", "error_flags")), (unpack, ("rows", "error_flags")),
                        (chunk, ("token_offsets", "seq_lens", "block_tables", "error_flags", "lse", "o", "q", "kv_pool", "workspace"))):
        for name in names:
            with pytest.raises(ValueError):
                call(**{name: ints})
    for call in (pack, unpack):
        with pytest.raises(ValueError):
            call(kv=bf)
