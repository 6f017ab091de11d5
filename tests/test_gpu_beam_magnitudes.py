"""A beam search's selection where logits are finite but large: masks by a finite value, padded vocabularies, logits far from
zero.  Against the definition in 64 bits; equal continuations go by beam, then token."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import search_plain as plain  # noqa: E402

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
LARGE = [1e7, 2.0 ** 24 - 1, 2.0 ** 24, 1e9, 4e9, 1e10, 1e12, 1e15, 1e20, 9e29, 3e38]
MASKS = [-1e7, -1e9, -4e9, -1e10, -1e12, -1e15, -1e20, -9e29, -3e38]


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_selection_primitive_amd as lib
    lib.load_library()
    return lib


def parts(beams, vocab):
    """Tokens of a part and parts of a row: 512 tokens, doubled until a search has 8192 parts at most."""
    chunk = 512
    while beams * -(-vocab // chunk) > 8192:
        chunk *= 2
    return chunk, -(-vocab // chunk)


def lse_bound(beams, vocab):
    """What log S may be off by, S the fp32 sum of e^(x - M) over a row, in units of u = 2^-24:

      33  of one lane's 32 terms: the exponential to 2 u, 31 additions (the other way of forming them, with the maximum's
          product in two parts: 2 u, 0.7 u of the argument, 2 u and u of the factor 2^-l, ten additions: less);
      2.3 ln V  of arguments: a difference d of logits or of maxima is rounded three times (itself, its product with log2 e,
          log2 e: u + u + 0.23 u) and errs by that times |d|, over all levels times |x - M|.  Weighted by e^(x - M) / S
          these are at most the entropy of the row, which is at most ln V;
      4 J of J joins one after the other, each an exponential (2 u), a product and an addition: the rest of a part's 512-token
          blocks, 16 lanes (4), the wave's other lanes (2), its workgroup's waves (3), the groups of 16 parts a lane reads
          after its first, and the lanes that hold any.

    1% for the products of errors."""
    chunk, chunks = parts(beams, vocab)
    groups = -(-chunks // 16)
    joins = chunk // 512 - 1 + 4 + 2 + 3 + -(-groups // 64) - 1 + math.ceil(math.log2(min(groups, 64)))
    return 1.01 * (33 + 2.3 * math.log(vocab) + 4 * joins) * 2.0 ** -24


def check(L, monkeypatch, logits, scores, k):
    monkeypatch.setattr(plain, "LSE", lse_bound(*logits.shape[1:]))
    got = L.beam_select(logits, scores, k)
    plain.check_selection(got, plain.continuations(logits, scores), logits, k)
    return got


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("value", LARGE + [-x for x in LARGE])
@pytest.mark.parametrize("vocab", [100, 5000])
def test_constant_rows(L, monkeypatch, vocab, value, dtype):
    logits = torch.full((2, 4, vocab), value, device="cuda", dtype=TYPES[dtype])
    s, parents, tokens = check(L, monkeypatch, logits, torch.zeros(2, 4, device="cuda"), 8)
    assert parents.tolist() == [[0] * 8] * 2 and tokens.tolist() == [list(range(8))] * 2
    assert (s + math.log(vocab)).abs().max() < 1e-5


def rows(seed, vocab, dtype, batch=2, beams=3):
    g = torch.Generator().manual_seed(seed)
    return ((3 * torch.randn(batch, beams, vocab, generator=g)).to(TYPES[dtype]).cuda(),
            (-5 * torch.rand(batch, beams, generator=g)).cuda())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("mask", MASKS)
def test_masks(L, monkeypatch, mask, dtype):
    """All but a few tokens, whole parts of 512, single lanes' tokens, in one beam and in all of a search."""
    for where in ("few are left", "parts", "a lane"):
        logits, scores = rows(1, 3000, dtype)
        hidden = torch.zeros(3000, dtype=torch.bool, device="cuda")
        if where == "few are left":
            hidden[:] = True
            hidden[[0, 5, 700, 701, 1535, 2047, 2999]] = False
        elif where == "parts":
            hidden[512:1536] = True
        else:  # the tokens 1024 .. 1535 of lane 3: every 16th run of 16 bytes
            run = 16 // logits.element_size()
            hidden[1024:1536] = torch.arange(512, device="cuda") // run % 16 == 3
        logits[0, 1, hidden] = mask
        logits[1, :, hidden] = mask
        _, parents, tokens = check(L, monkeypatch, logits, scores, 6)
        assert not hidden[tokens[1].long()].any(), where
        # a beam alone: it has to be there
        one = check(L, monkeypatch, logits[:1, 1:2].contiguous(), scores[:1, 1:2].contiguous(), 6)
        assert one[1].tolist() == [[0] * 6] and not hidden[one[2][0].long()].any(), where


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("mask", [-1e9, -1e10, -1e20])
def test_padded_vocabulary(L, monkeypatch, mask, dtype):
    """50257 tokens padded to 50304: the last part's last lanes hold padding alone."""
    logits, scores = rows(2, 50304, dtype, 1, 2)
    logits[:, :, 50257:] = mask
    check(L, monkeypatch, logits, scores, 8)


@pytest.mark.parametrize("offset", [1e8, -1e8, 1e11, -1e11])
def test_far_from_zero(L, monkeypatch, offset):
    """Logits that differ by whole steps of fp32 at a large offset."""
    logits, scores = rows(3, 2000, "fp32")
    step = 2.0 ** (math.floor(math.log2(abs(offset))) - 23)
    check(L, monkeypatch, offset + step * logits.round(), scores, 6)
