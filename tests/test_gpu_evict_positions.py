"""Eviction: which positions protect an entry, at the ends of the 32-bit range."""
import pytest

import test_gpu_cache as c

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
LOW, HIGH = -2 ** 31, 2 ** 31 - 1


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_selection_primitive_amd as lib
    lib.load_library()
    return lib


@pytest.mark.parametrize("capacity,keep", [(90, 40), (90, 89), (3000, 100), (20000, 6000), (20000, 19999)])
@pytest.mark.parametrize("recent", [0, 7])
def test_largest_position(L, capacity, keep, recent):
    """The largest position, as unfilled tables hold it, is protected by `recent` alone."""
    g = torch.Generator().manual_seed(capacity)
    positions = torch.argsort(torch.rand(1, 2, capacity, generator=g), 2).int()
    positions[0, 0, ::3] = HIGH
    positions[0, 1, 5:9] = HIGH
    c.check_evict(L, 1, 2, capacity, 16, [capacity], keep, positions=positions, sinks=2, recent=recent,
                  next_position=[HIGH])


@pytest.mark.parametrize("capacity,keep", [(90, 40), (20000, 6000)])
def test_without_next_position(L, capacity, keep):
    """No next_position: nothing but the sinks is protected."""
    a = torch.rand(1, 1, capacity, device="cuda") + 1.0
    p = torch.full((1, 1, capacity), HIGH, dtype=torch.int32, device="cuda")
    a[0, 0, :10] = 0.0  # the ten that leave first
    p[0, 0, 20:30] = 3
    a[0, 0, 20:30] = 0.0  # sinks
    k = torch.randn(1, 1, capacity, 16, device="cuda").bfloat16()
    n = torch.tensor([capacity], dtype=torch.int32, device="cuda")
    kept, _ = L.cache_evict(k, k.clone(), a.clone(), p, n, keep, sinks=4)
    got = set(kept[0, 0].tolist())
    assert not got & set(range(10)) and got >= set(range(20, 30))


@pytest.mark.parametrize("capacity,keep", [(90, 40), (20000, 6000)])
def test_smallest_next_position(L, capacity, keep):
    """next_position - recent below the 32-bit range: every entry is protected, and slots decide."""
    g = torch.Generator().manual_seed(3)
    positions = torch.randint(LOW, HIGH, (1, 1, capacity), generator=g, dtype=torch.int64).int()
    positions[0, 0, 0], positions[0, 0, 1] = LOW, HIGH
    c.check_evict(L, 1, 1, capacity, 16, [capacity], keep, positions=positions, recent=10, next_position=[LOW + 3])
