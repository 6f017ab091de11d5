"""What the cache operators write in place is known to autograd: a product that kept such a tensor for its backward
refuses instead of using the entries that took their place."""
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


@pytest.fixture(params=["native", "python"])
def front(request, L, monkeypatch):
    from sparse_selection_primitive_amd import hard
    L.dispatch_plan(torch.zeros(1, 1, dtype=torch.int32, device="cuda"), 1)  # binds
    if request.param == "native":
        if hard._native is None:
            pytest.skip("the native front is not built")
    else:
        monkeypatch.setattr(hard, "_native", None)
    return request.param


def arrays():
    k, v = (torch.randn(2, 2, 30, 64, device="cuda").bfloat16() for _ in range(2))
    a = torch.rand(2, 2, 30, device="cuda")
    p = torch.arange(30, dtype=torch.int32, device="cuda").expand(2, 2, 30).contiguous()
    return k, v, a, p, torch.tensor([30, 25], dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("what", ["k", "v", "account"])
def test_eviction_in_place_is_noticed(L, front, what):
    k, v, a, p, n = arrays()
    t = dict(k=k, v=v, account=a)[what]
    w = torch.ones_like(t).requires_grad_(True)
    y = (w * t).sum()  # keeps t for the gradient of w
    L.cache_evict(k, v, a, p, n, 20)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_attention_in_place_is_noticed(L, front):
    k, v, a, p, n = arrays()
    q = torch.randn(2, 1, 4, 64, device="cuda").bfloat16()
    w = torch.ones_like(a).requires_grad_(True)
    y = (w * a).sum()
    L.cache_attend(q, k, v, n, a)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_only_what_is_written_counts(L, front):
    """Inputs, and those of separate outputs, are as they were; the outputs are not."""
    k, v, a, p, n = arrays()
    q = torch.randn(2, 1, 4, 64, device="cuda").bfloat16()
    to, at = torch.zeros_like(a), torch.zeros_like(p)
    before, fresh = [t._version for t in (q, k, v, a, p, n)], to._version
    L.cache_attend(q, k, v, n, a, account_out=to)
    assert [t._version for t in (q, k, v, a, p, n)] == before and to._version == fresh + 1
    L.cache_evict(k, v, a, p, n, 20, account_out=to, positions_out=at)
    assert [t._version for t in (q, a, p, n)] == [before[i] for i in (0, 3, 4, 5)]
    assert k._version == before[1] + 1 and v._version == before[2] + 1
    assert to._version == fresh + 2
    assert at._version == fresh + 1


def test_inference_tensors(L, front):
    """Tensors made in inference mode have no versions, and are taken inside and outside of it."""
    with torch.inference_mode():
        k, v, a, p, n = arrays()
        q = torch.randn(2, 1, 4, 64, device="cuda").bfloat16()
        out = L.cache_attend(q, k, v, n, a)
        kept, _ = L.cache_evict(k, v, a, p, n, 20)
    k2, a2 = k.clone(), a.clone()
    L.cache_attend(q, k, v, n, a)
    L.cache_evict(k, v, a, p, n, 20)
    assert out.shape == q.shape and kept.shape == (2, 2, 20) and k2.shape == k.shape and a2.shape == a.shape


def test_outputs_of_the_caller_are_written(L):
    x, w = torch.randn(4, 16, device="cuda"), torch.rand(4, 2, device="cuda")
    weights, chosen = L.route_forward(x, 2)
    offsets, slot, _ = L.dispatch_plan(chosen, 16)
    xs = L.dispatch_forward(x, slot, offsets)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dys, dw = torch.empty_like(xs), torch.empty_like(w)
    before = [t._version for t in (weights, chosen, xs, y, dx, dys, dw)]
    L.route_forward(x, 2, out=(weights, chosen))
    L.route_backward(w, x, chosen, out=dx)
    L.dispatch_forward(x, slot, offsets, out=xs)
    L.dispatch_backward(xs, slot, out=dx)
    L.combine_forward(xs, slot, w, out=y)
    L.combine_backward(y, xs, slot, w, offsets, out=(dys, dw))
    after = [t._version for t in (weights, chosen, xs, y, dx, dys, dw)]
    assert [b - a for a, b in zip(before, after)] == [1, 1, 1, 1, 2, 1, 1]
