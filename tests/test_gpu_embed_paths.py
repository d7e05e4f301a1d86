"""The embedding's gradient where its two ways meet, counted and sorted tokens,
and where the sort of a large vocabulary looks at its tokens again. Against
float64 (tests/vocab_reference.py) and against each other."""
import numpy as np
import pytest

import vocab_reference as R
from gpu_common import dev, log
from ops_reference import check

pytestmark = pytest.mark.gpu


def _type(t):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[t]


@pytest.mark.parametrize("V", [163841, 600001])
def test_a_frequent_word_of_a_large_vocabulary(V):
    """More than 163840 words, and a word of four fifths of the tokens: more of a class in a wave's part of the ids
    (some 500) than it keeps (192)."""
    import torch
    import cross_entropy_amd as lm
    log(f"frequent word, V {V}")
    rng = np.random.default_rng(V)
    N, H = 10007, 24
    ids = rng.integers(0, V, N).astype(np.int32)
    ids[rng.random(N) < 0.8] = 77777
    ids[rng.random(N) < 0.05] = 77777 + 4096            # another word of its class
    ids[rng.random(N) < 0.05] = -1
    ids[0], ids[1] = 0, V - 1
    dy = rng.standard_normal((N, H)).astype(np.float32)
    rows = np.unique(ids[ids >= 0])
    at = torch.from_numpy(rows.astype(np.int64)).cuda()
    places = np.where(ids >= 0, np.searchsorted(rows, ids), -1)
    for old in (None, np.full((len(rows), H), 0.5, np.float32)):
        into = torch.full((V, H), float("nan") if old is None else 0.5, device="cuda")
        lm.embed_backward(dev(ids), dev(dy), dW=into, accumulate=old is not None)
        want, e = R.embed_grad(places, dy, len(rows), 1.0, old, "f32")
        check(into[at].cpu().numpy(), want, e, f"dW {V}")
        into[at] = 0.0 if old is None else 0.5
        assert bool((into == (0.0 if old is None else 0.5)).all())


@pytest.mark.parametrize("y,g", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("H", [72, 513])
def test_counted_and_sorted_tokens_give_the_same_bits(H, y, g):
    """2048 tokens are counted; the same with masked ones behind them are sorted. A word of 600 tokens, one of 33, one of
    32, and many of a few."""
    import torch
    import cross_entropy_amd as lm
    log(f"counted and sorted {H} {y} {g}")
    rng = np.random.default_rng(H)
    N, more, V = 2048, 300, 700
    ids = rng.integers(3, V, N).astype(np.int32)
    ids[:600], ids[600:633], ids[633:665] = 0, 1, 2
    ids = np.concatenate([rng.permutation(ids), np.full(more, -1, np.int32)])
    gen = torch.Generator(device="cuda").manual_seed(H)
    dy = torch.randn(N + more, H, device="cuda", generator=gen).to(_type(y))
    dy[N:] = float("nan")
    old = torch.randn(V, H, device="cuda", generator=gen).to(_type(g))
    d = dev(ids)
    for add in (False, True):
        few, many = (lm.embed_backward(d[:n], dy[:n], scale=3.7, dW=old.clone(), accumulate=add) for n in (N, N + more))
        assert torch.equal(few, many), add
        want, e = R.embed_grad(ids[:N], dy[:N].float().cpu().numpy(), V, 3.7, old.float().cpu().numpy() if add else None, g)
        check(many.float().cpu().numpy(), want, e, "dW")
