"""The two ways of the hard selections' binding: the native front, and the one written out in Python that takes every
call the front does not.  Both end in the same C calls, so their results are equal to the last bit; what the front does
not take (other strides, other types, mistakes) is converted or refused as without it."""
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_selection_primitive_amd as lib
    lib.load_library()
    return lib


@pytest.fixture()
def both(L, monkeypatch):
    from sparse_selection_primitive_amd import hard
    L.dispatch_plan(torch.zeros(1, 1, dtype=torch.int32, device="cuda"), 1)  # binds
    if hard._native is None:
        pytest.skip("the native front is not built")

    def run(f):
        fast = f()
        with monkeypatch.context() as m:
            m.setattr(hard, "_native", None)
            slow = f()
        return fast, slow
    return run


def same(a, b):
    a, b = (x if isinstance(x, tuple) else (x,) for x in (a, b))
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert x.dtype == y.dtype and x.shape == y.shape and x.is_contiguous() and not x.requires_grad
        assert torch.equal(x, y)


def test_built_front_is_used(L, both):
    from sparse_selection_primitive_amd import hard
    assert os.path.exists(hard._NATIVE_PATH)
    x = torch.randn(4, 16, device="cuda")
    assert hard._native.route_forward(x, None, 2, 0, 1, None, True, 1.0) is not None
    # not its to take
    assert hard._native.route_forward(x.cpu(), None, 2, 0, 1, None, True, 1.0) is None
    assert hard._native.route_forward(x.t(), None, 2, 0, 1, None, True, 1.0) is None
    assert hard._native.route_forward(x.double(), None, 2, 0, 1, None, True, 1.0) is None
    assert hard._native.route_forward(x, None, 99, 0, 1, None, True, 1.0) is None
    assert hard._native.route_forward(x, None, "2", 0, 1, None, True, 1.0) is None
    assert hard._native.route_forward(x) is None and hard._native.cache_evict(x) is None


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_route(L, both, dtype):
    x = torch.randn(100, 64, device="cuda").to(dtype)
    bias = torch.randn(64, device="cuda")
    dw = torch.randn(100, 6, device="cuda")
    for kw in (dict(), dict(score="sigmoid", scale=2.5), dict(renormalise=False)):
        same(*both(lambda: L.route_forward(x, 6, bias, groups=8, top_groups=3, **kw)))
        same(*both(lambda: L.route_forward(x[:, :40], 6, **kw)))  # rows at a distance
        same(*both(lambda: L.route_forward(x.t()[:, :50], 6, **kw)))  # columns: converted
        chosen = L.route_forward(x, 6, **kw)[1]
        same(*both(lambda: L.route_backward(dw, x, chosen, **kw)))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_dispatch(L, both, dtype):
    chosen = torch.randint(-1, 20, (70, 5), device="cuda", dtype=torch.int32)
    same(*both(lambda: L.dispatch_plan(chosen, 20)))
    big = torch.randint(0, 20, (700, 5), device="cuda", dtype=torch.int32)
    same(*both(lambda: L.dispatch_plan(big, 20)))
    offsets, slot, order = L.dispatch_plan(chosen, 20)
    x, dy = (torch.randn(70, 96, device="cuda").to(dtype) for _ in range(2))
    rows = torch.randn(350, 96, device="cuda").to(dtype)
    w = torch.rand(70, 5, device="cuda")
    for a in (x, torch.cat([x, x], 1)[:, :96], x.t().contiguous().t(), x[:1].expand(70, 96)):
        same(*both(lambda: L.dispatch_forward(a, slot, offsets)))
        same(*both(lambda: L.combine_backward(a, rows, slot, w, offsets)))
    for r in (rows, rows.t().contiguous().t()):
        same(*both(lambda: L.dispatch_backward(r, slot)))
        same(*both(lambda: L.combine_forward(r, slot, w)))
    same(*both(lambda: L.combine_forward(rows, slot.t().contiguous().t(), w.t().contiguous().t())))


@pytest.mark.parametrize("capacity", [100, 3000])
def test_cache(L, both, capacity):
    k, v = (torch.randn(2, 3, capacity, 64, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(2, 4, 6, 64, device="cuda").bfloat16()
    n = torch.tensor([capacity, capacity // 2], dtype=torch.int32, device="cuda")
    account = torch.rand(2, 3, capacity, device="cuda")
    positions = torch.arange(capacity, dtype=torch.int32, device="cuda").expand(2, 3, capacity).contiguous()
    for scale in (None, 0.3, 1):
        same(*both(lambda: L.cache_attend(q, k, v, n, scale=scale)))

    def attend():
        to = torch.zeros_like(account)
        return L.cache_attend(q, k, v, n, account, account_out=to), to

    def attend_in_place():
        to = account.clone()
        return L.cache_attend(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, n, to), to

    def evict():
        k2, v2, a2, p2 = k.clone(), v.clone(), account.clone(), positions.clone()
        kept, after = L.cache_evict(k2, v2, a2, p2, n, capacity // 3, next_position=n, sinks=2, recent=5)
        return kept, after, k2, v2, a2, p2

    def evict_apart():
        k2, v2, a2, p2 = k.clone(), v.clone(), torch.zeros_like(account), torch.zeros_like(positions)
        kept, after = L.cache_evict(k2, v2, account, positions, n, capacity - 1, account_out=a2, positions_out=p2)
        return kept, after, k2, v2, a2, p2
    for f in (attend, attend_in_place, evict, evict_apart):
        same(*both(f))


def test_refusals_do_not_depend_on_the_front(L, both):
    x = torch.randn(4, 16, device="cuda")
    k = torch.zeros(1, 1, 8, 64, device="cuda", dtype=torch.bfloat16)
    n = torch.tensor([8], dtype=torch.int32, device="cuda")
    a = torch.zeros(1, 1, 8, device="cuda")
    for bad in (lambda: L.route_forward(x, 0), lambda: L.route_forward(x, 2, score="none"),
                lambda: L.dispatch_plan(x, 4), lambda: L.cache_attend(k[:, :, 0], k, k, n),
                lambda: L.cache_attend(k, k, k, n, account_out=a), lambda: L.cache_evict(k, k, a, a.int(), n, 9)):
        def refused():
            with pytest.raises(L.LapsumError):
                bad()
            return torch.zeros(1)
        same(*both(refused))


def test_calls_on_another_stream_and_in_a_graph(L, both):
    x = torch.randn(64, 32, device="cuda")
    w, c = L.route_forward(x, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        w2, c2 = L.route_forward(x, 4)
    side.synchronize()
    same((w, c), (w2, c2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w3, c3 = L.route_forward(x, 4)
        offsets, slot, order = L.dispatch_plan(c3, 32)
    want = L.dispatch_plan(c, 32)
    for _ in range(3):
        w3.zero_(), c3.zero_(), slot.zero_()
        graph.replay()
        torch.cuda.synchronize()
        same((w, c), (w3, c3))
        same(want, (offsets, slot, order))


def test_integers_past_32_bits_are_refused_by_both_fronts(L, both):
    x = torch.randn(4, 16, device="cuda")
    k = torch.zeros(1, 1, 8, 64, device="cuda", dtype=torch.bfloat16)
    n, a = torch.tensor([8], dtype=torch.int32, device="cuda"), torch.zeros(1, 1, 8, device="cuda")
    for bad in (lambda: L.route_forward(x, 2 ** 32 + 2), lambda: L.route_forward(x, 2, groups=2 ** 32 + 1),
                lambda: L.cache_evict(k, k.clone(), a, a.int(), n, 4, sinks=2 ** 32),
                lambda: L.cache_evict(k, k.clone(), a, a.int(), n, 4, next_position=n, recent=2 ** 32 + 1)):
        def refused():
            with pytest.raises(L.LapsumError):
                bad()
            return torch.zeros(1)
        same(*both(refused))


def test_second_derivatives_are_refused(L):
    x = torch.randn(4, 16, device="cuda", requires_grad=True)
    w, c = L.route(x, 2)
    offsets, slot, _ = L.dispatch_plan(c, 16)
    y = L.combine(L.dispatch(x, slot, offsets), w, slot, offsets)
    g, = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
