"""The example of drafted decoding: its tokens are those of decoding one by one, in fewer
steps of the served model (drafting with the served model's own weights, every path of
the tree that follows it is kept)."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


def test_drafted_tokens_are_the_plain_ones():
    import drafted_decoding as d
    fq = d.fq
    weights = d.random_weights(3)
    served = d.Model(weights, lambda w: fq.W6AxLinear(w, abits=8))
    drafter = d.Model(weights, lambda w: fq.W4Linear(w, group=32))
    prompts = [[5, 400, 17], list(range(30)), [7]]
    plain, plain_steps = d.generate(served, prompts, 20)
    drafted, steps = d.generate(served, prompts, 20, drafter)
    assert drafted == plain and plain_steps == 20 and steps <= plain_steps
    again, own_steps = d.generate(served, prompts, 20, served)
    assert again == plain and own_steps <= 7
