"""What the Python calls of the 4-bit cache refuse before they reach the library, with arrays that stand in for
CUDA tensors and a library that only counts its calls (no GPU, nothing is launched)."""
import types

import pytest

torch = pytest.importorskip("torch")

import hierarchical_sparse_attention_gb300 as hs

A = 1 << 20  # an aligned stand-in address


class Array:
    """What the bindings ask of a CUDA tensor."""

    def __init__(self, device=0, dtype=torch.int32, stride=576):
        self.device_index, self.dtype, self.row = device, dtype, stride

    def get_device(self):
        return self.device_index

    def is_contiguous(self):
        return True

    def dim(self):
        return 2

    def size(self, i):
        return 8

    def stride(self, i):
        return (self.row, 1)[i]

    def data_ptr(self):
        return A


@pytest.fixture
def lib(monkeypatch):
    """The library's calls, counted, and the current device in `here`."""
    calls = types.SimpleNamespace(names=[], here=0)

    class Fake:
        def __getattr__(self, name):
            return lambda *a: calls.names.append(name) or 0

    monkeypatch.setattr(hs, "_lib", Fake())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: calls.here)
    return calls


def page_pool(x):
    return hs.make_page_pool([x], 4, 8, 100, 16, 416, x, x, x, x, x, 1 << 20, x)


PAGE_CALLS = [lambda p, x: hs.hs_pages_init(p), lambda p, x: hs.hs_pages_extend(p, 1, x, x, x, x),
              lambda p, x: hs.hs_pages_fork(p, 1, x, x, x, x), lambda p, x: hs.hs_pages_free(p, 1, x, x, x),
              lambda p, x: hs.hs_pages_compact(p)]


@pytest.mark.parametrize("call", PAGE_CALLS)
def test_a_page_pool_of_another_device_is_refused(lib, call):
    pool = page_pool(Array(0))
    call(pool, Array(0))
    assert len(lib.names) == 1
    lib.here = 1
    for entries in (Array(0), Array(1), A):  # the entries on either device, or raw
        with pytest.raises(ValueError):
            call(pool, entries)
    assert len(lib.names) == 1
    call(page_pool(Array(1)), Array(1))
    call(page_pool(A), A)  # addresses only: theirs to know
    assert len(lib.names) == 3


I, U, H, F, P = (Array(dtype=t) for t in (torch.int32, torch.uint32, torch.bfloat16, torch.float32, torch.uint8))
ROWS = dict(kv=H, rows=I, pool=P, err=I)
MLA = dict(q=H, pool=P, table=I, lens=I, o=H, lse=F, ws=P, err=I)
POOL = dict(pools=P, table=I, refs=I, free=I, count=I, err=I, ws=P)


def pack(kv, rows, pool, err):
    hs.hs_fp4_pack_rows(8, kv, 576, rows, 1.0, pool, 100, err)


def unpack(kv, rows, pool, err):
    hs.hs_fp4_unpack_rows(8, pool, 100, rows, 1.0, kv, 576, err)


def sparse(q, pool, table, lens, o, lse, ws, err):
    hs.hs_fp4_sparse_mla_decode(2, 16, 4, 1, q, pool, 100, table, 0.1, 1.0, o, lse, ws, 0, err)


def window(q, pool, table, lens, o, lse, ws, err):
    hs.hs_fp4_window_mla_decode(2, 16, 1, 8, 1, 1, q, pool, 100, 16, 8, lens, table, 0.1, 1.0, o, lse, ws, 0, err)


def make(pools, table, refs, free, count, err, ws):
    hs.hs_pages_init(hs.make_page_pool([pools], 4, 8, 100, 16, 416, table, refs, free, count, ws, 1 << 20, err))


def entries(a, b, c, granted):
    p = page_pool(A)
    hs.hs_pages_extend(p, 1, a, b, c, granted)
    hs.hs_pages_fork(p, 1, a, b, c, granted)


def ranges(a, b, c):
    hs.hs_pages_free(page_pool(A), 1, a, b, c)


@pytest.mark.parametrize("call,good", [(pack, ROWS), (unpack, ROWS), (sparse, MLA), (window, MLA), (make, POOL),
                                       (entries, dict(a=I, b=I, c=I, granted=I)), (ranges, dict(a=I, b=I, c=I))])
def test_arrays_of_another_type_are_refused(lib, call, good):
    """torch makes int64 where nothing else is asked for: read as 32-bit numbers, every second one is 0."""
    call(**good)
    call(**{k: U if v is I else v for k, v in good.items()})
    for bits in (torch.int16, torch.uint16):
        call(**{k: Array(dtype=bits) if v is H else v for k, v in good.items()})
    for name, of in good.items():
        call(**dict(good, **{name: A}))  # an address has no type
        if of is P:  # bytes of any kind
            call(**dict(good, **{name: Array(dtype=torch.int32)}))
            continue
        if call is sparse and name == "lens":
            continue
        for other in (torch.int64, torch.float16, torch.float64, torch.int8, torch.bool,
                      torch.float32 if of is not F else torch.int32, torch.int32 if of is H else torch.bfloat16):
            seen = len(lib.names)
            with pytest.raises(ValueError):
                call(**dict(good, **{name: Array(dtype=other)}))
            assert len(lib.names) == seen or call is entries


def test_addresses_need_no_torch():
    """The calls with raw addresses, in a process where torch cannot be imported."""
    import subprocess
    import sys
    code = ("import sys; sys.modules['torch'] = None\n"
            "import hierarchical_sparse_attention_gb300 as hs\nA = 1 << 20\n"
            "hs.hs_fp4_pack_rows(0, A, 576, A, 1.0, A, 100, A)\n"
            "hs.hs_fp4_sparse_mla_decode(0, 16, 64, 1, A, A, 100, A, 0.1, 1.0, A, A, None, 0, A)\n"
            "p = hs.make_page_pool([A], 4, 8, 100, 16, 416, A, A, A, A, A, hs.hs_pages_workspace_bytes(4, 100), A)\n"
            "hs.hs_pages_extend(p, 0, A, A, A)\nhs.hs_pages_fork(p, 0, None, None, None)\nhs.hs_pages_free(p, 0, A)\n")
    root = hs.__file__.rsplit("/", 2)[0]
    subprocess.run([sys.executable, "-c", code], cwd=root, check=True, timeout=120)
