"""The feed-forward operators together, as the example uses them: a layer
trains (its loss falls) and is served from E4M3 and 4-bit weights."""
import os
import sys

import pytest

from gpu_helpers import say

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_layer_trains_and_serves():
    import gated_ffn
    say("gated feed-forward example")
    got = gated_ffn.main(tokens=300, width=256, hidden=384, steps=25, log=say)
    losses, errors = got["losses"], got["errors"]
    assert losses[-1] < 0.7 * losses[0]
    assert all(b < 1.02 * a for a, b in zip(losses, losses[1:])), losses
    # root mean square roundings: E4M3 operands 2.6% each, so g and u 3.7%, h
    # about 6%, and with the quantized h and Wd 7%; 4-bit weights 10% (integers)
    # to 13% (E2M1) in each of three products, 18% to 24%
    assert errors["prompt"] < 0.12 and errors["int4"] < 0.3 and errors["mxfp4"] < 0.4, errors
