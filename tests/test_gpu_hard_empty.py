"""Calls without tokens, or without sequences, and sizes that nothing can be allocated for."""
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


def test_attend_without_new_tokens(L):
    """Nothing is added: account_out is account, in the filled entries."""
    k = torch.randn(3, 2, 40, 64, device="cuda").bfloat16()
    q = torch.empty(3, 0, 4, 64, device="cuda", dtype=torch.bfloat16)
    n = torch.tensor([40, -3, 17], dtype=torch.int32, device="cuda")
    account = torch.rand(3, 2, 40, device="cuda")
    before, to = account.clone(), torch.full_like(account, -7.0)
    out = L.cache_attend(q, k, k, n, account, account_out=to)
    assert out.shape == (3, 0, 4, 64) and torch.equal(account, before)
    there = torch.arange(40, device="cuda") < n[:, None, None].expand(3, 2, 1)
    assert torch.equal(to, torch.where(there, account, -7.0))
    assert L.cache_attend(q, k, k, n, account).shape == (3, 0, 4, 64) and torch.equal(account, before)
    assert L.cache_attend(q, k, k, n).shape == (3, 0, 4, 64)


@pytest.mark.parametrize("batch,heads", [(0, 2), (3, 0), (0, 0)])
def test_no_cache(L, batch, heads):
    k = torch.empty(batch, heads, 40, 64, device="cuda", dtype=torch.bfloat16)
    a = torch.empty(batch, heads, 40, device="cuda")
    n = torch.tensor([40, -3, 17][:batch], dtype=torch.int32, device="cuda")
    kept, after = L.cache_evict(k, k.clone(), a, a.int(), n, 20)
    assert kept.shape == (batch, heads, 20) and kept.dtype == torch.int32
    assert after.tolist() == [20, 0, 17][:batch] and after.dtype == torch.int32
    with pytest.raises(L.LapsumError):
        L.cache_evict(k, k.clone(), a, a.int(), n, 41)
    with pytest.raises(L.LapsumError):
        L.cache_evict(k, k.clone(), a, a.int(), n, 0)


@pytest.mark.parametrize("size", [2 ** 29, 2 ** 31, 2 ** 40, 2 ** 62, 2 ** 64 + 5, 10 ** 30])
def test_sizes_out_of_range_are_refused_before_anything_is_allocated(L, size):
    k = torch.zeros(64, 64, 8, 64, device="cuda", dtype=torch.bfloat16)
    a = torch.zeros(64, 64, 8, device="cuda")
    n = torch.full((64,), 8, dtype=torch.int32, device="cuda")
    x = torch.randn(4096, 16, device="cuda")
    c = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    held = torch.cuda.memory_allocated()
    for sign in (1, -1):
        for bad in (lambda: L.cache_evict(k, k, a, a.int(), n, sign * size), lambda: L.route_forward(x, sign * size),
                    lambda: L.dispatch_plan(c, sign * size), lambda: L.dispatch_plan(c[:0], sign * size)):
            with pytest.raises(L.LapsumError):
                bad()
    assert torch.cuda.max_memory_allocated() - held < 2 ** 20
