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
