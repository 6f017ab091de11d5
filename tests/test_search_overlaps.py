"""Outputs of the beam selection and the cache reordering in the memory of their inputs or of each other, refused by the C ABI
(no GPU): one search is read when another is written.  Device pointers are made-up addresses: every call ends in an argument
check."""
import os
import shutil
import subprocess

import pytest

import sparse_selection_primitive_amd as L
from sparse_selection_primitive_amd import hard

LAYOUT = 10
M = 1 << 24  # far apart


@pytest.fixture(scope="module")
def lib():
    return L.load_library()


BATCH, BEAMS, VOCAB, STRIDE, K = 3, 4, 100, 128, 8
BYTES = dict(logits=(BATCH * BEAMS - 1) * STRIDE * 4 + VOCAB * 4, scores=BATCH * BEAMS * 4, ended=BATCH * BEAMS, out=BATCH * K * 4,
             parents=BATCH * K * 4, tokens=BATCH * K * 4)
READ, WRITTEN = ("logits", "scores", "ended"), ("out", "parents", "tokens", "workspace")


def select(lib, **at):
    bytes_ = lib.lapsum_beam_select_workspace_bytes(BATCH, BEAMS, VOCAB, K)
    a = dict({n: (i + 1) * M for i, n in enumerate((*READ, *WRITTEN))}, **at)
    return lib.lapsum_beam_select(a["logits"], 0, BATCH, BEAMS, VOCAB, STRIDE, a["scores"], a["ended"], 2, K, a["out"],
                                  a["parents"], a["tokens"], a["workspace"], bytes_, None)


@pytest.mark.parametrize("one", WRITTEN)
@pytest.mark.parametrize("other", READ + WRITTEN)
def test_selection(lib, one, other):
    if one == other:
        return
    size = dict(BYTES, workspace=lib.lapsum_beam_select_workspace_bytes(BATCH, BEAMS, VOCAB, K))
    base = 64 * M
    step = 256 if one == "workspace" else 4  # it is aligned to as much
    for distance in {0, (size[other] - 1) // step * step, -((size[one] - 1) // step * step)}:  # the first, the last bytes
        assert -size[one] < distance < size[other]
        assert select(lib, **{other: base, one: base + distance}) == LAYOUT, distance


def test_rows_at_a_distance(lib):
    """The last row's own bytes count, wherever it is."""
    last = (BATCH * BEAMS - 1) * STRIDE * 4
    for at in (last, last + VOCAB * 4 - 4, 5 * STRIDE * 4 - 40):
        assert select(lib, out=M + at) == LAYOUT


def test_one_row(lib):
    """Of one row the distance to the next does not count, however large."""
    bytes_ = lib.lapsum_beam_select_workspace_bytes(1, 1, 50, 1)
    for stride in (50, 2 ** 40, 2 ** 63 - 1):
        assert lib.lapsum_beam_select(M, 0, 1, 1, 50, stride, 2 * M, None, 0, 1, M + 196, 3 * M, 4 * M, 5 * M, bytes_, None) == LAYOUT
    bytes_ = lib.lapsum_beam_select_workspace_bytes(1, 2, 50, 1)
    for stride in (50, 2 ** 40, 2 ** 63 - 1):
        assert lib.lapsum_beam_select(M, 0, 1, 2, 50, stride, 2 * M, None, 0, 1, M + 196, 3 * M, 4 * M, 5 * M, bytes_, None) == LAYOUT


# ------------------------------------------------------------ reordering
CACHES, HEADS, CAPACITY, WIDTH = 4, 2, 10, 16
ENTRY = 2 * WIDTH  # bytes
SIDE, PER_ENTRY = CACHES * HEADS * CAPACITY * ENTRY, CACHES * HEADS * CAPACITY * 4
ARRAYS = dict(k=SIDE, v=SIDE, account=PER_ENTRY, positions=PER_ENTRY, parents=CACHES * 4, lengths=CACHES * 4, after=CACHES * 4)
PACKED = (HEADS * CAPACITY * WIDTH, CAPACITY * WIDTH, WIDTH)  # strides of caches, heads and entries


def reorder(lib, ks=PACKED, vs=PACKED, size=(CACHES, HEADS, CAPACITY), **at):
    a = dict({n: (i + 1) * M for i, n in enumerate(ARRAYS)}, **at)
    c = hard.Cache(a["k"], a["v"], hard.BF16, WIDTH, *size, *ks, *vs)
    return lib.lapsum_cache_reorder(c, size[0], a["parents"], a["lengths"], a["account"], a["positions"], a["after"], None)


@pytest.mark.parametrize("one", ARRAYS)
@pytest.mark.parametrize("other", ARRAYS)
def test_reordering(lib, one, other):
    """Every pair but the two that are only read, and but keys that are the values."""
    if one == other or {one, other} == {"parents", "lengths"}:
        return
    base, step = 64 * M, 16 if one in "kv" else 4  # keys and values are aligned to 16 bytes
    distances = {0, (ARRAYS[other] - 1) // step * step, -((ARRAYS[one] - 1) // step * step)}
    for distance in distances - ({0} if {one, other} == {"k", "v"} else set()):
        assert -ARRAYS[one] < distance < ARRAYS[other]
        assert reorder(lib, **{other: base, one: base + distance}) == LAYOUT, distance


def test_keys_and_values_that_lie_unlike(lib):
    heads_last = (HEADS * CAPACITY * WIDTH, WIDTH, HEADS * WIDTH)
    wide = (HEADS * CAPACITY * 2 * WIDTH, CAPACITY * 2 * WIDTH, 2 * WIDTH)  # as much again between two entries
    for at in (0, 16, SIDE - 16, 16 - SIDE):
        assert reorder(lib, vs=heads_last, k=64 * M, v=64 * M + at) == LAYOUT
    # both with gaps, alike: the second half of an entry, entries further on
    for at in (16, -16, 2 * ENTRY, 5 * 2 * ENTRY + 16, 2 * SIDE - 2 * ENTRY, 2 * ENTRY - 2 * SIDE):
        assert reorder(lib, wide, wide, k=64 * M, v=64 * M + at) == LAYOUT, at
    # unlike, with gaps, from one place on; one without gaps between the entries of the other
    assert reorder(lib, wide, (wide[0], 2 * WIDTH, HEADS * 2 * WIDTH), k=64 * M, v=64 * M) == LAYOUT
    assert reorder(lib, wide, k=64 * M, v=64 * M + 16) == LAYOUT


def test_far_strides(lib):
    """Strides and sizes whose products pass 64 bits."""
    far = (2 ** 62, 2 ** 61, 2 ** 13)
    assert reorder(lib, far, far, (2, 2, 10), k=64 * M, v=64 * M + 16) == LAYOUT
    assert reorder(lib, far, far, (2, 2, 10), account=M + 9 * far[2] * 2) == LAYOUT


DRIVER = os.path.join(os.path.dirname(os.path.abspath(__file__)), "sanitize", "overlap_driver.cpp")


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(DRIVER), reason="needs g++ and the driver")
def test_against_sets_of_bytes(tmp_path):
    """Random small layouts: what is refused is what shares a byte (sanitizers on)."""
    exe = str(tmp_path / "overlaps")
    root = os.path.dirname(os.path.dirname(DRIVER)) + "/.."
    res = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                          "-D__HIP_PLATFORM_AMD__=1", "-I/opt/rocm/include", DRIVER,
                          os.path.join(root, "sparse_selection_primitive_amd", "csrc", "hard_api.cpp"), "-o", exe],
                         capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr
    res = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and "all checks passed" in res.stdout, res.stdout + res.stderr
