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
