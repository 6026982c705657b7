"""The example's language model: it learns its synthetic text with the library's gradients, and
its token-by-token form agrees with the parallel one."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu


def test_recurrent_lm_learns_and_steps():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import recurrent_lm as lm
    finally:
        sys.path.pop(0)
    print("example: training", flush=True)
    model, history = lm.train(steps=80, batch=16, length=193, vocab=127, dim=128, hidden=320, layers=1,
                              report=lambda s: print(s, flush=True))
    # uniform guessing costs log 127 = 4.84; copying costs about 0.1 log(127) + H(0.9) + the documents' starts
    assert history[0] > 4.0
    assert history[-1] < 0.6 * history[0], history
    # bf16 activations through a few roundings each way: 2^-8 each, of the largest logit
    assert lm.states_agree(model, 127) < 0.05
