"""The bound that the gradients of up to 64 tokens are held to, whose cotangent
is kept as two bf16 words: two words keep it, and one word, or a second word
with a fault, does not. On float64 values; the kernels are held to it in
tests/test_gpu_distill_few.py."""
import numpy as np
import pytest

import ops_reference as R
from synthetic import bf16_bits_to_f32, f32_to_bf16_bits
from test_gpu_distill import _case, _g

# tokens, H, vocabulary, entries: both paddings of up to 64 tokens, several splits of dh, ragged tiles
WORDS = [(1, 64, 5, 2), (9, 64, 17, 4), (32, 128, 40, 3), (33, 64, 70, 6), (50, 192, 19, 5), (64, 64, 300, 2)]


def words_case(N, H, V, K):
    return _case(60 + N, N, H, V, K, hard=True, pad=0.0)


def two_words(monkeypatch, N, V):
    """The bound's allowance for holding an entry: its rounding leaves at most
    2^-8 of it, whose own rounding leaves 2^-8 of that; and the products add
    twice as many terms, each 2^-24 of their sum at most."""
    monkeypatch.setitem(R.HALF, "bf16", 2.0 ** -16 + max(N, V) * R.U)


def _bf16(x):
    return bf16_bits_to_f32(f32_to_bf16_bits(x.astype(np.float32))).astype(np.float64)


@pytest.mark.parametrize("N,H,V,K", WORDS)
def test_two_words_and_no_less(N, H, V, K, monkeypatch):
    two_words(monkeypatch, N, V)
    h, W, targets, ids, t, tlse = words_case(N, H, V, K)
    ref = R.Distill(bf16_bits_to_f32(h), bf16_bits_to_f32(W), targets, ids, t, tlse, 1.0)
    g_kl, g_logp = _g(1, N, True)
    dh, dW, e_h, e_W = ref.backward(g_kl, g_logp, "f32")
    # the cotangent itself: the gradient of a table that is the identity
    eye = R.Distill.__new__(R.Distill)
    eye.__dict__ = dict(ref.__dict__, W=np.eye(V))
    dz = eye.backward(g_kl, g_logp, "f32")[0]
    assert np.allclose(dz @ ref.W, dh, rtol=1e-12, atol=1e-14)
    hi = _bf16(dz)
    lo = _bf16(dz - hi)

    def outside(x):
        return ((np.abs(x @ ref.W - dh) > e_h).any(), (np.abs(x.T @ ref.h - dW) > e_W).any())

    assert outside(hi + lo) == (False, False)
    faults = dict(one_word=hi, sign=hi - lo, twice=hi + 2 * lo, rows=hi + np.roll(lo, 1, 1))
    if N > 1:
        faults["tokens"] = hi + np.roll(lo, 1, 0)
    for name, x in faults.items():
        assert outside(x) == (True, True), name
