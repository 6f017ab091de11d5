"""Which layouts of a cache eviction writes into (argument checks of the C ABI: made-up addresses, nothing is launched;
a call that passes the layout check ends at the missing outputs)."""
import itertools

import pytest

import sparse_selection_primitive_amd as L
from sparse_selection_primitive_amd import hard

NULL, LAYOUT = 1, 10
P = 0x10000


@pytest.fixture(scope="module")
def lib():
    return L.load_library()


def refused(lib, shape, strides, which):
    batch, heads, capacity, width = shape
    free = (heads * capacity * width, capacity * width, width)
    k, v = (strides, free) if which == "k" else (free, strides)
    c = hard.Cache(P, P, hard.BF16, width, batch, heads, capacity, *k, *v)
    rc = lib.lapsum_cache_evict(c, None, P, P, 1, P, 0, 0, P, P, P, 2 * P, P, 2 ** 40, None)
    assert rc in (NULL, LAYOUT)
    return rc == LAYOUT


def meet(shape, strides):
    batch, heads, capacity, width = shape
    seen = set()
    for b, h, s in itertools.product(range(batch), range(heads), range(capacity)):
        at = b * strides[0] + h * strides[1] + s * strides[2]
        for e in range(at, at + width, 8):  # strides and widths are multiples of 8
            if e in seen:
                return True
            seen.add(e)
    return False


@pytest.mark.parametrize("which", ["k", "v"])
def test_entries_that_share_memory_are_refused(lib, which):
    steps = (0, 8, 16, 24, 32, 40, 48, 64, 96, 128, 160, 320)
    for shape in ((2, 2, 3, 16), (1, 3, 4, 8), (3, 1, 2, 24), (2, 3, 1, 16), (1, 1, 5, 16)):
        for strides in itertools.product(steps, repeat=3):
            if strides[2] >= shape[3] and meet(shape, strides):
                assert refused(lib, shape, strides, which), (shape, strides)


def test_the_usual_layouts_are_taken(lib):
    for batch, heads, capacity, width in ((2, 3, 10, 64), (1, 8, 1, 128), (4, 1, 7, 8), (1, 1, 1, 256)):
        shape = (batch, heads, capacity, width)
        w = width
        for strides in ((heads * capacity * w, capacity * w, w),           # head-major
                        (capacity * heads * w, w, heads * w),              # entry-major
                        (2 * heads * capacity * w, capacity * w, w),       # a slice, or keys beside values
                        (capacity * heads * 2 * w, 2 * w, heads * 2 * w),  # keys and values interleaved
                        (w, batch * w, heads * batch * w),                 # batch innermost
                        (heads * capacity * (w + 8), capacity * (w + 8), w + 8)):  # padded entries
            assert not refused(lib, shape, strides, "k") and not refused(lib, shape, strides, "v"), (shape, strides)
