"""Keys and values that are one tensor seen through two views, reordered on the GPU: moved once, equal to the last bit.  The
stride of a dimension of one place says nothing, and views differ in it."""
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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def views(kind, beams):
    """The tensor, its first view and another one of the same places."""
    if kind == "one head":
        x = torch.randn(beams, 500, 64, device="cuda").bfloat16()
        return x, x[:, None], x[:, :, None].transpose(1, 2)
    if kind == "one entry":
        x = torch.randn(beams, 40, 64, device="cuda").bfloat16()
        return x, x[:, :, None], x.as_strided((beams, 40, 1, 64), (40 * 64, 64, 512, 1))
    x = torch.randn(1, 3, 500, 64, device="cuda").bfloat16()  # one cache
    return x, x, x.as_strided(x.shape, (64, 500 * 64, 64, 1))


@pytest.mark.parametrize("front", ["native", "python"])
@pytest.mark.parametrize("kind,beams", [("one head", 4), ("one head", 20), ("one entry", 5), ("one cache", 1)])
def test_one_tensor_through_two_views(L, monkeypatch, kind, beams, front):
    from sparse_selection_primitive_amd import hard
    if front == "python":
        monkeypatch.setattr(hard, "_native", None)
    x, k, v = views(kind, beams)
    assert k.shape == v.shape and k.stride() != v.stride() and torch.equal(k, v)
    before, capacity = x.clone(), k.shape[2]
    for turn in range(1, 4):  # a ring: every cache changes places
        parents = i32([[(i + 1) % beams for i in range(beams)]])
        after = L.cache_reorder(k, v, parents, i32([capacity] * beams))
        assert after.tolist() == [capacity] * beams and torch.equal(x, before.roll(-turn, 0))


def test_entries_without_width_are_refused(L):
    """Accounts and positions have places then, which would have to move."""
    k, account = torch.zeros(2, 3, 8, 0, device="cuda").bfloat16(), torch.arange(48.0, device="cuda").view(2, 3, 8)
    before = account.clone()
    with pytest.raises(L.LapsumError):
        L.cache_reorder(k, k.clone(), i32([[1, 0]]), i32([8, 8]), account)
    assert torch.equal(account, before)
    # no cache, head or entry at all: there is nothing to move
    for shape in ((0, 3, 8, 64), (2, 0, 8, 64), (2, 3, 0, 64)):
        k = torch.zeros(shape, device="cuda").bfloat16()
        n = shape[0]
        assert L.cache_reorder(k, k.clone(), i32([[1, 0]]) if n else torch.zeros(0, 2, device="cuda", dtype=torch.int32),
                               i32([8, 5][:n])).tolist() == [min(5, shape[2]), min(8, shape[2])][:n]
