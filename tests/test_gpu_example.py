"""The example decoder end to end: prefill, token by token, and the same tokens as whole prompts."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_generate_agrees_with_prefill(gpu):
    import generate
    # Keys and values are off by half a unit in 127 of their page's largest, about 0.6% of a typical value, in each of 2 layers;
    # the residual stream carries the embedding unchanged: far less than 2% of the state's length, a cosine of 0.9998.
    # A wrong position, head or page changes an attention output altogether, a third of the state.
    assert generate.main(["--layers", "2", "--hidden", "1024", "--heads", "8", "--kv-heads", "2", "--ffn", "1024", "--new", "6",
                          "--batch", "3"]) > 0.995


def test_one_prompt_of_one_token(gpu):
    import generate
    model = generate.Decoder(1, 512, 4, 4, 512)
    tokens, states = model.generate([[7]], 3)
    assert tokens.shape == (1, 3) and states.shape == (3, 1, 512)
    assert generate.check(model, [[7]], tokens, states) > 0.995


def test_too_long_for_the_cache(gpu):
    import generate
    model = generate.Decoder(1, 512, 4, 4, 512, pages=4)
    with pytest.raises(ValueError, match="too small"):
        model.generate([[1] * 300], 3)
