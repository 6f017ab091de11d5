"""The beam search of examples/beam_decode.py: all operators of a decoder together.

With a budget that is never reached, every beam's cache has to hold the keys and values of its own history, and its score
has to be the sum of its tokens' log probabilities, both followed back through the parents.  Keys are products of
bf16 whose sum may be formed in another order, rounded once: they agree to a step, 2^-7 of their size; a
score of n steps to n times the bound of one selection and n roundings to fp32."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import search_plain as plain  # noqa: E402

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def E():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import beam_decode
    return beam_decode


@pytest.mark.parametrize("batch,beams", [(1, 4), (3, 5), (2, 1)])
def test_beams_keep_their_histories(E, batch, beams):
    s = E.Shape(batch=batch, prompt=20, budget=60, window=4)
    model = E.Model(s, vocab=700)
    g = torch.Generator(device="cuda").manual_seed(batch)
    prompt = torch.randint(3, 700, (batch, 20), generator=g, device="cuda")
    steps = 12
    with torch.no_grad():
        search = E.Search(model, prompt, beams)
        scores = search.scores.double()
        forked = 0
        for _ in range(steps):
            before, ended = scores, search.ended.clone()
            logits, parents = search.step()
            assert (parents >= 0).all()  # 700 tokens: there are always enough continuations
            forked += int((parents != torch.arange(beams, device="cuda")).sum())
            at = parents.long()
            logp = torch.log_softmax(logits.double(), 2)
            chosen = search.tokens[:, :, -1]
            step = logp[torch.arange(batch, device="cuda")[:, None], at, chosen]
            was = ended.gather(1, at)
            assert (chosen[was] == search.end_token).all()
            scores = before.gather(1, at) + torch.where(was, 0.0, step)
            assert ((scores - search.scores).abs() <= steps * (plain.LSE + 2.0 ** -24 * scores.abs())).all()
            assert (search.scores[:, 1:] <= search.scores[:, :-1]).all()
        assert beams == 1 or forked > 0
        # the caches: the prompt but its last token, then each beam's own tokens but the newest
        history = torch.cat([prompt[:, None, :-1].expand(batch, beams, 19), search.tokens[:, :, :-1]], 2)
        length = history.shape[2]
        assert search.cache.lengths.tolist() == [length] * (batch * beams)
        k, v = model.keys_values(model.embedding[history.reshape(batch * beams, length)])
        for got, want in ((search.cache.k, k), (search.cache.v, v)):
            got, want = got[:, :, :length].double(), want.double()
            assert ((got - want).abs() <= 2.0 ** -7 * want.abs() + 2.0 ** -9).all()
        where = torch.arange(length, device="cuda", dtype=torch.int32)
        assert (search.cache.positions[:, :, :length] == where).all()


def test_with_a_budget_and_ends(E):
    s = E.Shape(batch=2, prompt=80, budget=32, window=8, sinks=2, recent=8)
    model = E.Model(s, vocab=50)
    model.embedding[2] *= 1.5  # the end comes up
    g = torch.Generator(device="cuda").manual_seed(9)
    with torch.no_grad():
        search = E.Search(model, torch.randint(3, 50, (2, 80), generator=g, device="cuda"), 6)
        for _ in range(40):
            search.step()
    assert search.cache.lengths.tolist() == [32] * 12 and (search.scores > -torch.inf).all()
    for b in range(12):
        for h in range(s.kv_heads):
            held = set(search.cache.positions[b, h, :32].tolist())
            assert len(held) == 32 and held >= {0, 1} | set(range(79 + 40 - 8, 79 + 40))


def test_main(E, capsys):
    search = E.main(["--steps", "6", "--beams", "3"])
    assert torch.isfinite(search.scores).all() and "6 steps" in capsys.readouterr().out
