"""The example that trains a token model with the library's operators: the loss
starts at that of random logits over the vocabulary and falls as the model
learns the permutation it is shown."""
import math
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,vocab,dim", [(2048, 256, 64), (4096, 512, 128)])
def test_training_learns_the_permutation(tokens, vocab, dim):
    import train_tokens
    losses = train_tokens.train(steps=40, tokens=tokens, vocab=vocab, dim=dim)
    assert all(math.isfinite(x) for x in losses)
    assert math.log(vocab) - 0.5 < losses[0] < math.log(vocab) + 1.5
    assert losses[-1] < 0.1 * losses[0]
