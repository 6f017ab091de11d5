"""Outputs of the beam selection in the memory of its inputs or of each other, refused by the C ABI (no GPU): one search is
read when another is written.  Device pointers are made-up addresses: every call ends in an argument check."""
import pytest

import sparse_selection_primitive_amd as L

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
