"""Caches that follow the beams of a search, on the GPU: equal to the last bit."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import search_plain as plain  # noqa: E402


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_selection_primitive_amd as lib
    lib.load_library()
    return lib


def state(caches, heads, capacity, width, dtype=torch.bfloat16, extra=True):
    out = dict(k=torch.randn(caches, heads, capacity, width, device="cuda").to(dtype),
               v=torch.randn(caches, heads, capacity, width, device="cuda").to(dtype))
    if extra:
        out["account"] = torch.rand(caches, heads, capacity, device="cuda")
        out["positions"] = torch.randint(0, 999, (caches, heads, capacity), device="cuda", dtype=torch.int32)
    return out


def call(L, s, parents, lengths):
    return L.cache_reorder(s["k"], s["v"], parents, lengths, s.get("account"), s.get("positions"))


def check(L, s, parents, lengths):
    want, after = plain.reorder(s, parents, lengths)
    got = call(L, s, parents, lengths)
    assert got.dtype == torch.int32 and got.cpu().tolist() == after.tolist()
    for n in s:
        assert torch.equal(s[n], want[n]), n


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("parents", [[0, 1, 2, 3], [0, 0, 0, 0], [3, 3, 3, 3], [1, 0, 3, 2], [1, 2, 3, 0], [2, 2, 0, 0],
                                     [-1, 0, 4, 1], [-1, -1, -1, -1]])
@pytest.mark.parametrize("extra", [False, True])
def test_maps(L, parents, extra):
    for lengths in ([70, 70, 70, 70], [0, 1, 33, 100], [100, 200, -3, 64]):
        check(L, state(4, 2, 100, 64, extra=extra), i32([parents]), i32(lengths))


@pytest.mark.parametrize("beams", [1, 2, 4, 5, 8, 9, 16, 17, 40, 64])
@pytest.mark.parametrize("width", [8, 96, 256])
def test_beams(L, beams, width):
    g = torch.Generator().manual_seed(beams)
    parents = torch.randint(-1 if beams > 1 else 0, beams, (3, beams), generator=g, dtype=torch.int32).cuda()
    lengths = torch.randint(0, 80, (3 * beams,), generator=g, dtype=torch.int32).cuda()
    check(L, state(3 * beams, 2, 77, width, torch.float16), parents, lengths)


@pytest.mark.parametrize("capacity,heads", [(1, 1), (31, 3), (32, 1), (33, 8), (1000, 2), (4097, 1)])
def test_capacities(L, capacity, heads):
    parents = torch.randint(0, 4, (2, 4), device="cuda", dtype=torch.int32)
    lengths = torch.randint(0, capacity + 1, (8,), device="cuda", dtype=torch.int32)
    check(L, state(8, heads, capacity, 128), parents, lengths)


def test_layouts(L):
    """Heads and entries changed over, entries at a distance, keys and values of one tensor; arrays of the same kind."""
    parents, lengths = i32([[1, 1, 0], [2, 0, 1]]), i32([50, 60, 20, 60, 60, 5])
    for make in (lambda: torch.randn(6, 60, 2, 64, device="cuda").bfloat16().transpose(1, 2),
                 lambda: torch.randn(6, 2, 60, 192, device="cuda").bfloat16()[..., 64:128],
                 lambda: torch.randn(2, 60, 6, 64, device="cuda").bfloat16().permute(2, 0, 1, 3),
                 lambda: torch.randn(12, 2, 60, 64, device="cuda").bfloat16()[::2]):
        s = dict(k=make(), v=make())
        base = s["k"]._base.clone() if s["k"]._base is not None else None
        check(L, s, parents, lengths)
        assert base is not None
    both = torch.randn(6, 2, 60, 2, 64, device="cuda").bfloat16()
    check(L, dict(k=both[..., 0, :], v=both[..., 1, :]), parents, lengths)


@pytest.mark.parametrize("name", ["account", "positions"])
def test_one_of_the_arrays(L, name):
    s = state(4, 2, 300, 64)
    check(L, {n: s[n] for n in ("k", "v", name)}, i32([[1, 1, 3, 2]]), i32([300, 290, 5, 257]))


@pytest.mark.parametrize("beams", [3, 12, 20])
def test_keys_that_are_the_values(L, beams):
    k = torch.randn(beams, 2, 70, 64, device="cuda").bfloat16()
    want, after = plain.reorder(dict(k=k), i32([[(i + 1) % beams for i in range(beams)]]), i32([70] * beams))
    got = L.cache_reorder(k, k, i32([[(i + 1) % beams for i in range(beams)]]), i32([70] * beams))
    assert got.tolist() == after.tolist() and torch.equal(k, want["k"])


def test_twice_in_a_row_and_versions(L):
    s, lengths = state(4, 2, 50, 64), i32([50, 40, 30, 20])
    versions = {n: x._version for n, x in s.items()}
    check(L, s, i32([[1, 2, 3, 0]]), lengths)
    assert all(s[n]._version > versions[n] for n in s)
    check(L, s, i32([[3, 3, 1, 1]]), i32([40, 30, 20, 50]))


def test_past_32_bits(L):
    """A cache whose last sequences lie past 2^32 bytes."""
    if torch.cuda.mem_get_info()[0] < 40 * 2 ** 30:
        pytest.skip("needs 40 GiB")
    n, capacity = 4, 300000
    k = torch.zeros(n, 16, capacity, 128, device="cuda", dtype=torch.bfloat16)  # 1.2 GB a beam
    for i in range(n):
        k[i, 15, capacity - 1] = i + 1
        k[i, 3, 200000] = 10 * (i + 1)
    after = L.cache_reorder(k, k.clone(), i32([[3, 2, 1, 0]]), i32([capacity] * 4))
    assert after.tolist() == [capacity] * 4
    assert k[:, 15, capacity - 1, 5].tolist() == [4, 3, 2, 1] and k[:, 3, 200000, 0].tolist() == [40, 30, 20, 10]


def test_nothing_to_do(L):
    k = torch.zeros(0, 2, 8, 64, device="cuda").bfloat16()
    assert L.cache_reorder(k, k.clone(), torch.zeros(0, 2, device="cuda", dtype=torch.int32), i32([])).shape == (0,)
    k = torch.zeros(4, 0, 8, 64, device="cuda").bfloat16()
    assert L.cache_reorder(k, k.clone(), i32([[1, 0], [-1, 1]]), i32([3, 9, 5, 6])).tolist() == [8, 3, 0, 6]


def test_refusals(L):
    s, lengths = state(4, 2, 50, 64), i32([50, 40, 30, 20])
    parents = i32([[1, 0], [0, 1]])
    for bad in (dict(k=s["k"].float(), v=s["v"].float()), dict(v=s["v"][:2]), dict(v=s["v"].half()),
                dict(k=s["k"][:1].expand(4, 2, 50, 64)), dict(account=s["account"].double()),
                dict(account=s["account"].transpose(1, 2).contiguous().transpose(1, 2)), dict(positions=s["positions"].long()),
                dict(positions=s["positions"][:2]), dict(k=s["k"].cpu())):
        with pytest.raises(L.LapsumError):
            call(L, dict(s, **bad), parents, lengths)
    for p in (i32([[0, 1, 2]]), parents.long(), parents.flatten(), parents.cpu(), i32([[0, 1]])):
        with pytest.raises(L.LapsumError):
            call(L, s, p, lengths)
    for n in (lengths.long(), lengths[:2], lengths.cpu()):
        with pytest.raises(L.LapsumError):
            call(L, s, parents, n)


def test_both_fronts_streams_and_graph(L, monkeypatch):
    from sparse_selection_primitive_amd import hard
    s, lengths, parents = state(8, 2, 90, 64), i32([90, 80, 70, 60, 9, 0, 7, 6]), i32([[1, 2, 3, 0], [1, 1, 0, 0]])
    start = {n: x.clone() for n, x in s.items()}
    want, after = plain.reorder(s, parents, lengths)

    def again():
        for n in s:
            s[n].copy_(start[n])

    def same(got):
        torch.cuda.synchronize()
        assert got.tolist() == after.tolist() and all(torch.equal(s[n], want[n]) for n in s)
    with monkeypatch.context() as m:
        m.setattr(hard, "_native", None)
        same(call(L, s, parents, lengths))
    again()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call(L, s, parents, lengths)
    same(got)
    again()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(L, s, parents, lengths)
    for _ in range(3):
        again()
        graph.replay()
        same(got)
