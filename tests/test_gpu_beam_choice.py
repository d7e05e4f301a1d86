"""The beam step's choice where float32 does not decide it: masks with bits set
past the vocabulary, words of vanishing probability beside beams that are held
back or of another row's large logits, allowed words far below the largest one.
Against float64 (tests/vocab_reference.py)."""
import numpy as np
import pytest

import vocab_reference as R
from gpu_common import dev, dev_bits, log
from synthetic import bf16_bits_to_f32, f32_to_bf16_bits

pytestmark = pytest.mark.gpu


def _run(h, W, scores, allowed, G, C):
    import cross_entropy_amd as lm
    out = lm.beam_step(dev_bits(h), dev_bits(W), dev(scores), G, C, None, dev(allowed))
    return [x.cpu().numpy() for x in out]


def _reference(h, W, scores, allowed, G, C):
    return R.Beams(bf16_bits_to_f32(h), bf16_bits_to_f32(W), scores, G, C, None, allowed)


def _bits(words, N, V):
    """Masks of N rows that allow the given words."""
    a = np.zeros((N, -(-V // 32)), np.uint32)
    np.bitwise_or.at(a, (slice(None), words >> 5), np.uint32(1) << (words & 31).astype(np.uint32))
    return a.view(np.int32)


# the tiles (more than 256 rows) and the streaming kernels; vocabularies that end inside a mask's word
@pytest.mark.parametrize("B,G,V,C", [(24, 16, 4001, 40), (40, 8, 30011, 20), (2, 16, 4001, 40)])
@pytest.mark.parametrize("far", [-1e4, -1e9])
def test_mask_bits_past_the_vocabulary(B, G, V, C, far):
    """The bits of words that do not exist mean nothing: a row may have them set where its last real words are forbidden."""
    log(f"mask tail {B} {G} {V} {far}")
    rng = np.random.default_rng(V + B)
    N, H = B * G, 64
    W = f32_to_bf16_bits((0.1 * rng.standard_normal((V, H))).astype(np.float32))
    h = f32_to_bf16_bits(rng.standard_normal((N, H)).astype(np.float32))
    scores = np.full((B, G), far, np.float32)
    scores[:, 0] = -12.0                            # one beam, the others held back at two distances
    scores[:, 2::3] *= 0.75
    allowed = np.full((N, -(-V // 32)), -1, np.int32)
    allowed[::G] = _bits(np.array([3, 1000, 2000]), 1, V)
    allowed[::G, -1] = np.uint32(0xFFFFFFFF << (V % 32) & 0xFFFFFFFF).view(np.int32)
    case = (h, W, scores.reshape(N), allowed, G, C)
    _reference(*case).check(*_run(*case), f"{B} x {G}, V {V}, {far}")


@pytest.mark.parametrize("B", [1, 16, 80])
@pytest.mark.parametrize("far", [-1e6, -1e9])
def test_words_of_vanishing_probability(B, far):
    """A leading beam that may take a few words, and others of logit -1e30 (a padded vocabulary): the held-back beams'
    words lie between the two, and are ordered by their own logits."""
    log(f"vanishing words {B} {far}")
    rng = np.random.default_rng(B)
    G, C, H, V = 4, 20, 64, 8000
    N = B * G
    # small whole numbers, whose logits are exact in any order, but for the last 500 words
    h = rng.integers(-3, 4, (N, H)).astype(np.float32)
    W = rng.integers(-2, 3, (V, H)).astype(np.float32) / 16
    h[:, 0], W[:, 0], W[-500:, 0] = 1.0, 0.0, -1e30
    scores = np.tile(np.array([-5.0, 0.75 * far, far, -np.inf], np.float32), B)
    allowed = np.full((N, -(-V // 32)), -1, np.int32)
    allowed[::G] = _bits(np.concatenate([[7, 1500, 3000], np.arange(V - 400, V)]), 1, V)
    case = (f32_to_bf16_bits(h), f32_to_bf16_bits(W), scores, allowed, G, C)
    want, got = _reference(*case), _run(*case)
    # equal logits are equal scores in 64 bits, others at least 1 / 16 apart: the words are the very same ones
    assert np.array_equal(got[1], want.ids) and np.array_equal(got[2], want.parents)


@pytest.mark.parametrize("B", [1, 16, 80])
def test_far_rows_beside_a_row_of_large_logits(B):
    """What is far for a row of ordinary logits is not made near by another row's large ones: the leading beam's reach
    some 5e5, the next ones are held back by 1e8, where float32 has steps of 8."""
    log(f"far beside large {B}")
    rng = np.random.default_rng(B)
    G, C, H, V = 4, 20, 64, 8000
    N = B * G
    h = rng.integers(-3, 4, (N, H)).astype(np.float32)
    W = rng.integers(-2, 3, (V, H)).astype(np.float32) / 16
    h[::G] *= 2.0 ** 17
    scores = np.tile(np.array([-5.0, -7.5e7, -1e8, -np.inf], np.float32), B)
    allowed = np.full((N, -(-V // 32)), -1, np.int32)
    allowed[::G] = _bits(np.array([7, 1500, 3000]), 1, V)
    case = (f32_to_bf16_bits(h), f32_to_bf16_bits(W), scores, allowed, G, C)
    want, got = _reference(*case), _run(*case)
    assert np.array_equal(got[1], want.ids) and np.array_equal(got[2], want.parents)


@pytest.mark.parametrize("N", [16, 64, 300])
def test_allowed_words_far_below_the_largest_logit(N):
    """The largest logit lies near 0 and is forbidden; the allowed words lie near -3000, where float32 has steps of
    2.4e-4, and a few of them within each step: the order is that of 64 bits all the same."""
    log(f"far below {N}")
    rng = np.random.default_rng(N)
    H, V, C = 256, 2000, 8
    h = (0.05 * rng.standard_normal((N, H))).astype(np.float32)
    W = (0.01 * rng.standard_normal((V, H))).astype(np.float32)
    h[:, 0], W[:, 0], W[::2, 0] = 64.0, 0.0, -47.0
    case = (f32_to_bf16_bits(h), f32_to_bf16_bits(W), np.full(N, -1.0, np.float32), _bits(np.arange(0, V, 2), N, V), 1, C)
    want, got = _reference(*case), _run(*case)
    # the reference's logits are sums of products of 16 bits between 2^12 and some 2^-40, off by 2^-41 at most; the best
    # nine lie further apart than that
    best = np.sort(want.found, 1)[:, -C - 1:]
    assert np.diff(best, axis=1).min() > 2.0 ** -38
    assert np.array_equal(got[1], want.ids)
