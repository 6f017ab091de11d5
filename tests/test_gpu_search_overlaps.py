"""Arrays that lie next to each other, or between rows of another, without sharing memory: accepted by the C ABI, with the
results of arrays of their own."""
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


@pytest.mark.parametrize("batch", [1, 3])
def test_selection_in_one_buffer(L, batch):
    lib, stream = L.load_library(), torch.cuda.current_stream().cuda_stream
    beams, vocab, stride, k = 4, 100, 128, 7
    places, need = batch * k, lib.lapsum_beam_select_workspace_bytes(batch, beams, vocab, k)
    g = torch.Generator().manual_seed(0)
    x, scores = torch.randn(batch, beams, vocab, generator=g).cuda(), -torch.rand(batch, beams, generator=g).cuda()
    want = L.beam_select(x, scores, k)
    # the workspace, the logits, then what is written between the logits' rows or behind them
    head = (need + 255) // 256 * 64
    buffer = torch.full((head + batch * beams * stride + 4 * places + 64,), float("nan"), device="cuda")
    rows = buffer[head:head + batch * beams * stride].view(batch * beams, stride)
    rows[:, :vocab] = x.view(-1, vocab)
    behind = buffer[head + (batch * beams - 1) * stride + vocab:]
    behind[3 * places:3 * places + batch * beams] = scores.flatten()
    at = [behind.data_ptr() + 4 * i * places for i in range(3)]
    if 4 * places <= 4 * (stride - vocab):
        at[2] = rows[1, vocab:].data_ptr()  # between two rows
    assert lib.lapsum_beam_select(rows.data_ptr(), 0, batch, beams, vocab, stride, behind[3 * places:].data_ptr(), None, 0, k, *at,
                                  buffer.data_ptr(), need, stream) == 0
    torch.cuda.synchronize()
    base = buffer.data_ptr()
    got = [buffer[(p - base) // 4:(p - base) // 4 + places].view(batch, k) for p in at]
    assert torch.equal(got[0], want[0])
    assert torch.equal(got[1].view(torch.int32), want[1]) and torch.equal(got[2].view(torch.int32), want[2])


@pytest.mark.parametrize("kind", ["halves of an entry", "one after the other", "by cache", "by token", "a third", "heads last"])
def test_caches_in_one_tensor(L, kind):
    """Keys and values woven into one tensor without meeting."""
    n, h, c, w = 4, 2, 60, 64
    shape, side = {
        "halves of an entry": ((n, h, c, 2, w), lambda x, i: x[..., i, :]),
        "one after the other": ((2, n, h, c, w), lambda x, i: x[i]),
        "by cache": ((n, 2, h, c, w), lambda x, i: x[:, i]),
        "by token": ((n, c, 2, h, w), lambda x, i: x[:, :, i].transpose(1, 2)),
        "a third": ((n, c, 3, h, w), lambda x, i: x[:, :, i + 1].transpose(1, 2)),
        "heads last": ((c, n, h, 2 * w), lambda x, i: x[..., i * w:(i + 1) * w].permute(1, 2, 0, 3)),
    }[kind]
    x = torch.randn(shape, device="cuda").bfloat16()
    before = x.clone()
    parents, lengths = torch.tensor([[1, 0, 0, 2]], dtype=torch.int32), torch.tensor([60, 50, 9, 0], dtype=torch.int32)
    after = L.cache_reorder(side(x, 0), side(x, 1), parents.cuda(), lengths.cuda())
    assert after.tolist() == [50, 60, 60, 9]
    want = before.clone()
    for i in range(2):
        for j, p in enumerate(parents[0].tolist()):
            m = int(lengths[p])
            side(want, i)[j, :, :m] = side(before, i)[p, :, :m]
    assert torch.equal(x, want)


def test_arrays_behind_one_another(L):
    """Keys, values, accounts, positions, parents and lengths in one buffer, end to end."""
    n, h, c, w = 4, 2, 60, 64
    side, entries = n * h * c * w // 2, n * h * c  # words
    buffer = torch.randint(0, 2 ** 14, (2 * side + 2 * entries + 2 * n,), device="cuda", dtype=torch.int32)
    parts = torch.split(buffer, [side, side, entries, entries, n, n])
    k, v = (p.view(torch.bfloat16).view(n, h, c, w) for p in parts[:2])
    account, positions = parts[2].view(torch.float32).view(n, h, c), parts[3].view(n, h, c)
    parts[4].copy_(torch.tensor([1, 1, 3, 0])), parts[5].copy_(torch.tensor([60, 31, 0, 7]))
    before = [x.view(torch.int32).clone() for x in (k, v, account, positions)]
    after = L.cache_reorder(k, v, parts[4].view(1, n), parts[5], account, positions)
    assert after.tolist() == [31, 31, 7, 60]
    for x, was in zip((k, v, account, positions), before):
        want = was.clone()
        for j, (p, m) in enumerate([(1, 31), (1, 31), (3, 7), (0, 60)]):
            want[j, :, :m] = was[p, :, :m]
        assert torch.equal(x.view(torch.int32), want)
