"""A beam search's selection on the GPU against its definition in 64 bits."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import search_plain as plain  # noqa: E402

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_selection_primitive_amd as lib
    lib.load_library()
    return lib


def inputs(batch, beams, vocab, dtype="fp32", seed=0, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    logits = (spread * torch.randn(batch, beams, vocab, generator=g)).to(TYPES[dtype]).cuda()
    scores = (-10 * torch.rand(batch, beams, generator=g)).cuda()
    return logits, scores


def check(L, logits, scores, k=None, ended=None, end_token=None):
    got = L.beam_select(logits, scores, k, ended=ended, end_token=end_token)
    want = plain.continuations(logits, scores, ended, end_token)
    plain.check_selection(got, want, logits, logits.shape[1] if k is None else k)
    return got


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 100, 511, 512, 513, 1000, 8192, 8193, 32001])
def test_vocabularies(L, vocab, dtype):
    check(L, *inputs(2, 3, vocab, dtype), 6)


@pytest.mark.parametrize("batch,beams,k", [(1, 1, 1), (1, 1, 64), (3, 2, 5), (5, 64, 64), (2, 17, 34), (70, 4, 8)])
def test_beams(L, batch, beams, k):
    check(L, *inputs(batch, beams, 1200, "bf16"), k)


def test_default_k(L):
    got = check(L, *inputs(2, 5, 300))
    assert got[0].shape == (2, 5)


def test_fewer_continuations_than_places(L):
    logits, scores = inputs(2, 2, 5)
    got = check(L, logits, scores, 30)
    assert (got[1][:, 10:] == -1).all()


@pytest.mark.parametrize("value", [0.0, -math.inf, -3e38, 3e38, -65504.0, 1e-30])
@pytest.mark.parametrize("vocab", [100, 5000])
def test_constant_rows(L, vocab, value):
    """Everything equal (more candidates than the list holds): the lowest places, in order.  Only masks: none."""
    logits = torch.full((2, 4, vocab), value, device="cuda")
    scores = torch.zeros(2, 4, device="cuda")
    s, parents, tokens = check(L, logits, scores, 8)
    if value > -math.inf:
        assert parents.tolist() == [[0] * 8] * 2 and tokens.tolist() == [list(range(8))] * 2
        assert (s + math.log(vocab)).abs().max() < 1e-5
    else:
        assert (parents == -1).all() and (tokens == -1).all() and (s == -math.inf).all()


def test_constant_rows_of_many_beams(L):
    """More equal parts than the list holds."""
    logits = torch.zeros(1, 64, 20000, device="cuda").bfloat16()
    scores = torch.zeros(1, 64, device="cuda")
    scores[0, :5] = -1.0
    _, parents, tokens = check(L, logits, scores, 20)
    assert parents.tolist() == [[5] * 20] and tokens.tolist() == [list(range(20))]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_many_ties(L, dtype):
    g = torch.Generator().manual_seed(1)
    logits = torch.randint(0, 3, (3, 4, 6000), generator=g).to(TYPES[dtype]).cuda()
    logits[1, 1] = logits[1, 0]  # equal rows with equal scores: ties between beams
    scores = torch.tensor([[-1.0, -2.0, -3.0, -4.0], [-1.0, -1.0, -5.0, -5.0], [0.0, 0.0, 0.0, 0.0]], device="cuda")
    check(L, logits, scores, 16)
    # equal beams, the best token once each: the beams in order
    logits = torch.zeros(1, 4, 900, device="cuda")
    logits[:, :, 700] = 5.0
    _, parents, tokens = check(L, logits, torch.zeros(1, 4, device="cuda"), 4)
    assert parents.tolist() == [[0, 1, 2, 3]] and tokens.tolist() == [[700] * 4]


def test_masked_infinite_and_nan(L):
    logits, scores = inputs(8, 3, 2000)
    logits[0, :, 10:] = -math.inf         # few tokens are left
    logits[1, 0] = -math.inf              # a beam without any
    logits[2, 1, 7] = math.nan            # a beam that is not a distribution
    logits[3, 0, [5, 600, 1999]] = math.inf  # they share it
    logits[4, 2] = math.inf
    logits[5, 0, :1990] = -3.4e38         # the type's lowest value as a mask
    logits[6, :, :] = math.nan            # nothing is left
    logits[7, 1, 3], logits[7, 1, 900] = math.inf, math.nan
    scores[1, 1] = -math.inf              # no beam
    scores[2, 2] = math.nan
    scores[4, 0] = math.inf
    s, parents, tokens = check(L, logits, scores, 6)
    assert (parents[6] == -1).all()
    assert sorted(tokens[3][parents[3] == 0].tolist()) == [5, 600, 1999] or scores[3, 0] < scores[3].max()
    assert 1 not in parents[1].tolist() and 0 not in parents[1].tolist()


def test_first_step(L):
    """The first step of a search: one beam lives."""
    logits, scores = inputs(3, 4, 700)
    scores[:, 1:] = -math.inf
    scores[:, 0] = 0.0
    _, parents, _ = check(L, logits, scores, 8)
    assert (parents == 0).all()


@pytest.mark.parametrize("end", [0, 511, 512, 1299])
def test_ended_beams(L, end):
    logits, scores = inputs(6, 4, 1300, "bf16")
    ended = torch.zeros(6, 4, dtype=torch.bool, device="cuda")
    ended[0, 0] = ended[1, :3] = ended[2] = ended[4, 3] = True
    logits[1, 0] = math.nan  # not read
    scores[4, 3] = -math.inf
    s, parents, tokens = check(L, logits, scores, 8, ended, end)
    assert sorted(parents[2].tolist()) == [-1] * 4 + [0, 1, 2, 3] and (tokens[2][:4] == end).all()
    for b, p, t in zip(range(6), parents.tolist(), tokens.tolist()):
        for i, j, value in zip(p, t, s[b].tolist()):
            if i >= 0 and bool(ended[b, i]):
                assert j == end and value == float(scores[b, i])


def test_far_apart(L):
    """Scores and logits of very different sizes: no overflow, beams of tiny probability last."""
    logits, scores = inputs(3, 3, 1500, spread=1.0)
    logits[0] *= 1e4
    logits[1] += 1e30
    logits[2] *= 1e37
    scores[0, 0], scores[0, 1] = -1e6, -1e-6
    check(L, logits, scores, 5)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_layouts(L, dtype):
    logits, scores = inputs(4, 3, 1001, dtype)
    want = check(L, logits, scores, 6)
    wide = torch.full((4, 3, 1010), math.nan, device="cuda", dtype=logits.dtype)
    views = [wide[:, :, 3:1004], wide[:, :, :1001]]
    apart = torch.full((4, 5, 1001), math.nan, device="cuda", dtype=logits.dtype)[:, 1:4]
    swapped = torch.empty(3, 4, 1001, device="cuda", dtype=logits.dtype).transpose(0, 1)
    columns = torch.empty(4, 1001, 3, device="cuda", dtype=logits.dtype).transpose(1, 2)
    for x in (*views, apart, swapped, columns):
        x.copy_(logits)
        got = L.beam_select(x, scores, 6)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    one = L.beam_select(logits[:, 1:2], scores[:, 1:2], 6)
    assert all(torch.equal(a, b) for a, b in zip(one, L.beam_select(logits[:, 1:2].contiguous(), scores[:, 1:2], 6)))
    assert L.beam_select(logits[:0], scores[:0], 6)[0].shape == (0, 6)


def test_large_vocabulary_and_long_rows(L):
    check(L, *inputs(1, 64, 150000, "bf16"), 64)  # parts of more than 512 tokens
    check(L, *inputs(1, 2, 2 ** 20, "fp16"), 10)


def test_refusals(L):
    x, s = inputs(2, 3, 50)
    e = torch.zeros(2, 3, dtype=torch.bool, device="cuda")
    for bad in (lambda: L.beam_select(x, s, 0), lambda: L.beam_select(x, s, 65), lambda: L.beam_select(x[0], s, 2),
                lambda: L.beam_select(x, s[:1], 2), lambda: L.beam_select(x, s.double(), 2),
                lambda: L.beam_select(x.double(), s, 2), lambda: L.beam_select(x, s, 2, ended=e),
                lambda: L.beam_select(x, s, 2, ended=e, end_token=50), lambda: L.beam_select(x, s, 2, ended=e, end_token=-1),
                lambda: L.beam_select(x, s, 2, ended=e.int(), end_token=1), lambda: L.beam_select(x, s.cpu(), 2),
                lambda: L.beam_select(x[:, :0], s[:, :0], 2), lambda: L.beam_select(x[:, :, :0], s, 2),
                lambda: L.beam_select(torch.zeros(1, 65, 4, device="cuda"), torch.zeros(1, 65, device="cuda"), 2),
                lambda: L.beam_select(x, s, 2 ** 32 + 2), lambda: L.beam_select(x, s, 2, ended=e, end_token=2 ** 32)):
        with pytest.raises(L.LapsumError):
            bad()


def test_both_fronts_streams_and_graph(L, monkeypatch):
    from sparse_selection_primitive_amd import hard
    x, s = inputs(3, 4, 3000, "bf16")
    e = torch.rand(3, 4, device="cuda") < 0.3

    def run():
        return L.beam_select(x, s, 8, ended=e, end_token=2)
    want = run()
    with monkeypatch.context() as m:
        m.setattr(hard, "_native", None)
        assert all(torch.equal(a, b) for a, b in zip(run(), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(3):
        for y in got:
            y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        x.neg_(), s.copy_(s.flip(1))
        want = run()
