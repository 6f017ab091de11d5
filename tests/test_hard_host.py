"""Host logic of the hard selections (no GPU): argument checks through the C ABI, workspace sizes, struct layouts.
Device pointers here are made-up addresses: every call ends in an argument check, nothing is launched."""
import ctypes

import pytest

import sparse_selection_primitive_amd as L
from sparse_selection_primitive_amd import hard

OK, NULL, SHAPE, WORKSPACE, OPTION, LAYOUT = 0, 1, 2, 5, 7, 10
P = 0x10000  # 256-byte aligned


@pytest.fixture(scope="module")
def lib():
    return L.load_library()


def options(**kw):
    base = dict(k=2, score=0, groups=1, top_groups=1, renormalise=1, scale=1.0)
    return hard.RouteOptions(*dict(base, **kw).values())


def cache(**kw):
    base = dict(k=P, v=P, dtype=hard.BF16, width=64, batch=2, heads=2, capacity=100, kb=12800, kh=6400, ke=64,
                vb=12800, vh=6400, ve=64)
    return hard.Cache(*dict(base, **kw).values())


def test_struct_sizes():
    assert ctypes.sizeof(hard.RouteOptions) == 6 * 4
    assert ctypes.sizeof(hard.Cache) == 2 * 8 + 2 * 4 + 9 * 8


def test_status_string_of_the_layout_error(lib):
    assert lib.lapsum_status_string(LAYOUT).decode() != "unknown status"


def test_route_checks(lib):
    def fwd(opt, dtype=0, tokens=4, experts=16, stride=16, logits=P, weights=P, chosen=P):
        return lib.lapsum_route_forward(logits, dtype, tokens, experts, stride, None, opt, weights, chosen, None)

    def bwd(opt, **kw):
        a = dict(dw=P, logits=P, dtype=0, tokens=4, experts=16, stride=16, chosen=P, out=P, **kw)
        return lib.lapsum_route_backward(a["dw"], a["logits"], a["dtype"], a["tokens"], a["experts"], a["stride"],
                                         a["chosen"], opt, a["out"], None)

    for call in (fwd, bwd):
        for bad in (dict(k=0), dict(k=17), dict(k=33), dict(score=2), dict(score=-1), dict(groups=0), dict(groups=3),
                    dict(groups=4, top_groups=0), dict(groups=4, top_groups=5), dict(renormalise=2),
                    dict(scale=float("nan")), dict(scale=float("inf"))):
            assert call(options(**bad)) == OPTION, bad
        assert call(None) == NULL
    assert fwd(options(), dtype=3) == OPTION and fwd(options(), dtype=-1) == OPTION
    assert fwd(options(), tokens=0) == SHAPE and fwd(options(), tokens=2 ** 24 + 1) == SHAPE
    assert fwd(options(), experts=0) == SHAPE and fwd(options(), experts=1025, stride=1025) == SHAPE
    assert fwd(options(), stride=15) == LAYOUT
    assert fwd(options(groups=128), experts=1024, stride=1024) == OPTION
    for missing in ("logits", "weights", "chosen"):
        assert fwd(options(), **{missing: None}) == NULL


def test_dispatch_checks(lib):
    def plan(chosen=P, tokens=4, k=2, experts=8, offsets=P, slot=P, order=P, ws=None, nbytes=0):
        return lib.lapsum_dispatch_plan(chosen, tokens, k, experts, offsets, slot, order, ws, nbytes, None)

    assert plan(tokens=0) == SHAPE and plan(k=0) == SHAPE and plan(k=33) == SHAPE and plan(experts=0) == SHAPE
    assert plan(experts=1025) == SHAPE and plan(tokens=2 ** 22 + 1) == SHAPE
    for missing in ("chosen", "offsets", "slot", "order"):
        assert plan(**{missing: None}) == NULL
    need = lib.lapsum_dispatch_plan_workspace_bytes(5000, 4, 64)
    assert need > 0 and lib.lapsum_dispatch_plan_workspace_bytes(16, 8, 1024) == 0
    assert lib.lapsum_dispatch_plan_workspace_bytes(0, 4, 64) == 0
    assert plan(tokens=5000, k=4, experts=64) == NULL
    assert plan(tokens=5000, k=4, experts=64, ws=P, nbytes=need - 1) == WORKSPACE
    assert plan(tokens=5000, k=4, experts=64, ws=P + 16, nbytes=need) == WORKSPACE

    calls = {
        "forward": lambda x=P, dtype=0, tokens=4, k=2, width=8, stride=8, slot=P, out=P:
            lib.lapsum_dispatch_forward(x, dtype, tokens, k, width, stride, slot, P, 8, out, None),
        "backward": lambda x=P, dtype=0, tokens=4, k=2, width=8, slot=P, out=P:
            lib.lapsum_dispatch_backward(x, dtype, tokens, k, width, slot, out, None),
        "combine": lambda x=P, dtype=0, tokens=4, k=2, width=8, slot=P, out=P:
            lib.lapsum_combine_forward(x, dtype, tokens, k, width, slot, P, out, None),
        "combine backward": lambda x=P, dtype=0, tokens=4, k=2, width=8, stride=8, slot=P, out=P:
            lib.lapsum_combine_backward(x, stride, P, dtype, tokens, k, width, slot, P, P, 8, out, P, None),
    }
    for name, call in calls.items():
        assert call(dtype=3) == OPTION, name
        assert call(tokens=0) == SHAPE and call(k=0) == SHAPE and call(k=40) == SHAPE and call(width=0) == SHAPE, name
        assert call(x=None) == NULL and call(slot=None) == NULL and call(out=None) == NULL, name
    assert calls["forward"](stride=7) == LAYOUT and calls["combine backward"](stride=7) == LAYOUT
    assert lib.lapsum_dispatch_forward(P, 0, 4, 2, 8, 8, P, P, 0, P, None) == SHAPE


def test_attend_checks(lib):
    def call(c, q=P, lengths=P, news=1, heads=4, scale=0.125, account=P, account_out=P, out=P, ws=P, nbytes=2 ** 40):
        return lib.lapsum_cache_attend(q, c, lengths, news, heads, scale, account, account_out, out, ws, nbytes, None)

    for bad, want in ((dict(dtype=hard.F32), OPTION), (dict(width=0), SHAPE), (dict(width=12), SHAPE),
                      (dict(width=264), SHAPE), (dict(batch=0), SHAPE), (dict(heads=0), SHAPE),
                      (dict(heads=2 ** 24), SHAPE), (dict(capacity=0), SHAPE), (dict(capacity=2 ** 30 + 1), SHAPE),
                      (dict(ke=60), LAYOUT), (dict(vb=-8), LAYOUT), (dict(k=None), NULL), (dict(v=P + 8), LAYOUT)):
        assert call(cache(**bad)) == want, bad
    c = cache()
    assert call(None) == NULL
    assert call(c, news=0) == SHAPE and call(c, heads=3) == SHAPE and call(c, heads=0) == SHAPE
    assert call(c, news=65536, heads=4) == SHAPE
    assert call(c, scale=float("nan")) == OPTION
    assert call(c, q=P + 2) == LAYOUT and call(c, out=P + 2) == LAYOUT
    assert call(c, q=None) == NULL and call(c, lengths=None) == NULL and call(c, out=None) == NULL
    assert call(c, account=None) == NULL and call(c, account_out=None) == NULL
    assert lib.lapsum_cache_attend_workspace_bytes(c, 1, 4, 1) == 0  # short caches need none
    long = cache(capacity=100000, kh=6400000, kb=12800000, vh=6400000, vb=12800000)
    need = lib.lapsum_cache_attend_workspace_bytes(long, 1, 4, 1)
    assert need >= lib.lapsum_cache_attend_workspace_bytes(long, 1, 4, 0) > 0
    assert call(long, nbytes=need - 1) == WORKSPACE and call(long, ws=P + 8) == WORKSPACE
    assert call(long, ws=None) == NULL
    assert lib.lapsum_cache_attend_workspace_bytes(cache(width=4), 1, 4, 1) == 0


def test_evict_checks(lib):
    def call(c, account=P, positions=P, lengths=P, keep=10, nxt=P, sinks=0, recent=0, account_out=P, positions_out=P,
             kept=P, lengths_out=2 * P, ws=P, nbytes=2 ** 40):
        return lib.lapsum_cache_evict(c, account, positions, lengths, keep, nxt, sinks, recent, account_out,
                                      positions_out, kept, lengths_out, ws, nbytes, None)

    c = cache()
    assert call(c, keep=0) == SHAPE and call(c, keep=101) == SHAPE
    assert call(c, sinks=-1) == OPTION and call(c, recent=-1) == OPTION
    assert call(c, recent=1, nxt=None) == NULL
    for missing in ("account", "positions", "lengths", "account_out", "positions_out", "kept", "lengths_out"):
        assert call(c, **{missing: None}) == NULL
    assert call(c, lengths_out=P) == LAYOUT
    for bad in (dict(ke=56), dict(ve=0), dict(kh=0), dict(vb=0), dict(k=P + 8)):
        assert call(cache(**bad)) == LAYOUT, bad
    assert call(cache(dtype=hard.F32)) == OPTION and call(None) == NULL
    assert lib.lapsum_cache_evict_workspace_bytes(c, 10) == 0  # short rows need none
    long = cache(capacity=100000, kh=6400000, kb=12800000, vh=6400000, vb=12800000)
    need = lib.lapsum_cache_evict_workspace_bytes(long, 10)
    assert need > 0 and lib.lapsum_cache_evict_workspace_bytes(long, 100001) == 0
    assert call(long, nbytes=need - 1) == WORKSPACE and call(long, ws=None) == NULL


def test_no_cpu_path():
    import torch
    x = torch.zeros(2, 4)
    for call in (lambda: L.route_forward(x, 1), lambda: L.dispatch_plan(x.int(), 4),
                 lambda: L.cache_attend(x, x, x, x), lambda: L.cache_evict(x, x, x, x, x, 1)):
        with pytest.raises(L.LapsumError):
            call()


def test_the_first_call_may_be_a_differentiable_one(monkeypatch):
    import torch
    monkeypatch.setattr(hard, "torch", None)  # as before any call
    x = torch.zeros(2, 4)
    for call in (lambda: L.route(x, 1), lambda: L.dispatch(x, x, x), lambda: L.combine(x, x, x, x)):
        with pytest.raises(L.LapsumError):
            call()
        hard.torch = None


def test_integers_past_32_bits_are_refused():
    with pytest.raises(L.LapsumError):
        hard._route_options(2 ** 32 + 2, "softmax", 1, 1, True, 1.0)
    with pytest.raises(L.LapsumError):
        hard._route_options(2, "softmax", 2 ** 32 + 1, None, True, 1.0)
    with pytest.raises(L.LapsumError):
        hard._int32(-2 ** 31 - 1, "sinks")
    assert hard._int32(2 ** 31 - 1, "recent") == 2 ** 31 - 1
