"""Host logic of the experts' products, the beam selection and the cache reordering (no GPU): argument checks through
the C ABI, workspace sizes, struct layouts, and what the Python side refuses without a device.  Device pointers are
made-up addresses: every call ends in an argument check, nothing is launched."""
import ctypes

import pytest

import sparse_selection_primitive_amd as L
from sparse_selection_primitive_amd import hard

OK, NULL, SHAPE, WORKSPACE, OPTION, LAYOUT = 0, 1, 2, 5, 7, 10
P = 0x10000


@pytest.fixture(scope="module")
def lib():
    return L.load_library()


def experts(**kw):
    base = dict(w=P, dtype=hard.BF16, reserved=0, experts=4, inputs=16, outputs=24, se=384, si=24, so=1)
    return hard.Experts(*dict(base, **kw).values())


def test_struct_sizes():
    assert ctypes.sizeof(hard.Experts) == 8 + 2 * 4 + 6 * 8


def products(lib):
    def forward(w, x=16 * P, stride=16, rows=10, offsets=P, out=32 * P):
        return lib.lapsum_expert_product_forward(x, stride, rows, w, offsets, out, None)

    def rows_(w, x=16 * P, stride=24, rows=10, offsets=P, out=32 * P):
        return lib.lapsum_expert_product_backward_rows(x, stride, rows, w, offsets, out, None)

    def weights(w, x=16 * P, stride=16, rows=10, offsets=P, out=32 * P, dy_stride=24):
        return lib.lapsum_expert_product_backward_weights(x, stride, out, dy_stride, rows, offsets, w, None)
    return forward, rows_, weights


def test_product_checks(lib):
    for call in products(lib):
        assert call(None) == NULL
        for bad, want in ((dict(dtype=3), OPTION), (dict(dtype=-1), OPTION), (dict(experts=0), SHAPE), (dict(experts=1025), SHAPE),
                          (dict(inputs=0), SHAPE), (dict(outputs=0), SHAPE),
                          (dict(inputs=2 ** 20 + 1, so=1, si=24), SHAPE), (dict(si=23), LAYOUT), (dict(so=2), LAYOUT),
                          (dict(si=1, so=15), LAYOUT), (dict(si=1, so=1), LAYOUT), (dict(si=2 ** 21 + 1), LAYOUT),
                          (dict(se=-1), LAYOUT), (dict(w=None), NULL)):
            assert call(experts(**bad)) == want, bad
        assert call(experts(), rows=0) == SHAPE and call(experts(), rows=2 ** 23 + 1) == SHAPE
        for missing in ("x", "offsets", "out"):
            assert call(experts(), **{missing: None}) == NULL
        assert call(experts(), stride=15) == LAYOUT and call(experts(), stride=2 ** 21 + 1) == LAYOUT
        assert call(experts(w=32 * P)) == LAYOUT  # in one place with what the call writes, or reads
    for call in products(lib)[:2]:
        assert call(experts(), out=16 * P) == LAYOUT and call(experts(), out=16 * P + 100) == LAYOUT
    weights = products(lib)[2]
    assert weights(experts(), dy_stride=23) == LAYOUT
    assert weights(experts(se=383)) == LAYOUT and weights(experts(se=0)) == LAYOUT  # matrices that share memory


def test_beam_checks(lib):
    def call(x=P, dtype=0, batch=2, beams=4, vocab=100, stride=100, scores=2 * P, ended=None, end=-1, k=4, out=P, parents=P,
             tokens=P, ws=P, nbytes=2 ** 40):
        return lib.lapsum_beam_select(x, dtype, batch, beams, vocab, stride, scores, ended, end, k, out, parents, tokens,
                                      ws, nbytes, None)

    assert call(dtype=3) == OPTION and call(dtype=-1) == OPTION
    for bad in (dict(batch=0), dict(beams=0), dict(beams=65), dict(vocab=0), dict(vocab=2 ** 20 + 1, stride=2 ** 21),
                dict(batch=2 ** 24)):
        assert call(**bad) == SHAPE, bad
    assert call(k=0) == OPTION and call(k=65) == OPTION
    assert call(stride=99) == LAYOUT and call(scores=P) == LAYOUT
    assert call(ended=P) == OPTION and call(ended=P, end=100) == OPTION
    for missing in ("x", "scores", "out", "parents", "tokens"):
        assert call(**{missing: None}) == NULL
    need = lib.lapsum_beam_select_workspace_bytes(2, 4, 100, 4)
    assert need > 0 and lib.lapsum_beam_select_workspace_bytes(2, 4, 100, 65) == 0
    assert call(nbytes=need - 1) == WORKSPACE and call(ws=None) == NULL and call(ws=P + 8) == WORKSPACE
    # the parts of a row do not grow past what one workgroup looks through
    assert lib.lapsum_beam_select_workspace_bytes(1, 64, 2 ** 20, 4) <= 8192 * 8


def test_reorder_checks(lib):
    def cache(**kw):
        base = dict(k=P, v=P, dtype=hard.BF16, width=64, batch=4, heads=2, capacity=100, kb=12800, kh=6400, ke=64,
                    vb=12800, vh=6400, ve=64)
        return hard.Cache(*dict(base, **kw).values())

    def call(c, beams=2, parents=P, lengths=P, account=P, positions=P, after=2 * P):
        return lib.lapsum_cache_reorder(c, beams, parents, lengths, account, positions, after, None)

    c = cache()
    assert call(None) == NULL
    assert call(c, beams=0) == SHAPE and call(c, beams=3) == SHAPE and call(c, beams=65) == SHAPE
    assert call(cache(batch=65), beams=65) == SHAPE
    for bad in (dict(dtype=hard.F32),):
        assert call(cache(**bad)) == OPTION
    for bad in (dict(ke=56), dict(ve=0), dict(kh=0), dict(vb=0), dict(k=P + 8), dict(ke=60)):
        assert call(cache(**bad)) == LAYOUT, bad
    for missing in ("parents", "lengths", "after"):
        assert call(c, **{missing: None}) == NULL
    assert call(c, after=P) == LAYOUT


def test_no_cpu_path():
    import torch
    x, w = torch.zeros(4, 8).bfloat16(), torch.zeros(2, 8, 8).bfloat16()
    o, n = torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    c = torch.zeros(4, 2, 8, 8).bfloat16()
    for call in (lambda: L.expert_product(x, w, o), lambda: L.expert_product_forward(x, w, o),
                 lambda: L.expert_product_backward(x, x, w, o), lambda: L.beam_select(torch.zeros(1, 2, 9), torch.zeros(1, 2)),
                 lambda: L.cache_reorder(c, c, n.view(2, 2), n)):
        with pytest.raises(L.LapsumError):
            call()


def test_plain_forms_agree_with_differences():
    """The reference's gradients against central differences of its products (linear: the difference is exact)."""
    import torch

    import search_plain as plain
    g = torch.Generator().manual_seed(0)
    xs, dys = torch.randn(9, 5, generator=g).double(), torch.randn(9, 4, generator=g).double()
    w, offsets = torch.randn(3, 5, 4, generator=g).double(), torch.tensor([1, 4, 4, 8])
    _, dxs, dw = plain.products(xs, w, offsets, dys)

    def value(x, m):
        return float((plain.products(x, m, offsets)[0][0] * dys).sum())
    for i in range(9):
        for j in range(5):
            d = torch.zeros_like(xs)
            d[i, j] = 0.5
            assert abs(value(xs + d, w) - value(xs - d, w) - float(dxs[0][i, j])) < 1e-9
    for e in range(3):
        for i in range(5):
            for j in range(4):
                d = torch.zeros_like(w)
                d[e, i, j] = 0.5
                assert abs(value(xs, w + d) - value(xs, w - d) - float(dw[0][e, i, j])) < 1e-9
