"""The fp32 sum of exponentials of a beam search's selection on rows whose parts' maxima ascend by small steps, so that nearly
all of the sum is brought to another maximum at every join: against 64 bits, to the bound of the longest chain of joins."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from test_gpu_beam_magnitudes import TYPES, lse_bound  # noqa: E402


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_selection_primitive_amd as lib
    lib.load_library()
    return lib


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("step", [1e-6, 1e-4, 3e-3, 0.1])
@pytest.mark.parametrize("beams,vocab", [(2, 40000), (2, 2 ** 20), (64, 2 ** 20)])
@pytest.mark.parametrize("level", [0.0, 5.0])
def test_ascending_maxima(L, beams, vocab, step, level, dtype):
    k = 5
    # a step from each run of 32 tokens to the next: those are what lanes, parts and workgroups hold, in some order
    run = torch.arange(vocab, dtype=torch.float64).div(32, rounding_mode="floor") * step
    row = torch.stack([run, run.flip(0)]) * (512 / vocab if step == 0.1 else 1) + level
    live = row.to(TYPES[dtype])
    logits = torch.full((1, beams, vocab), float("nan"), device="cuda", dtype=TYPES[dtype])  # of beams without a score
    scores = torch.full((1, beams), -torch.inf, device="cuda")
    # scores that the sum's logarithm takes away again: what is left is small, and so is its rounding
    logits[0, :2], scores[0, :2] = live.cuda(), (torch.logsumexp(live.double(), 1) - live.double().amax(1)).float().cuda()
    got, parents, tokens = (x.cpu()[0] for x in L.beam_select(logits, scores, k))
    want = torch.log_softmax(live.double(), 1) + scores[0, :2].double().cpu()[:, None]
    bound = lse_bound(beams, vocab)
    assert (parents >= 0).all() and (parents < 2).all()
    theirs = want[parents.long(), tokens.long()]
    err = (got.double() - theirs).abs() - 2.0 ** -24 * theirs.abs()
    print(f"beams {beams} vocab {vocab} step {step} level {level} {dtype}: off by {float(err.max()) * 2 ** 24:.2f} of "
          f"{bound * 2 ** 24:.0f} x 2^-24")
    assert err.max() <= bound
    assert (theirs >= want.flatten().topk(k).values - 2 * bound).all()
    assert len({(int(p), int(t)) for p, t in zip(parents, tokens)}) == k
