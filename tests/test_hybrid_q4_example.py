"""GPU test of the hybrid decoder with rotated queries and keys and with the 4-bit cache: the same prompts in one step
and in chunks give the same last logits.

Tolerances.  With a bf16 cache that of test_hybrid_example.py, whose derivation holds with one more rounding a layer
(the rotation's): sqrt(4 x 9) 2^-8 = 2.3e-2.  With a 4-bit cache a key or value that differs by bf16's rounding, d = 2^-8
of its size x, falls on the other side of a border between codes with probability d x / s, and then differs by s: its
mean square difference is d x s, for x of about 0.8 and s of about 0.4 deviations 2^-8 x 0.32, 0.035 of the deviation
in the root.  Up to four such differences (a key, a value, in two decoders) in a layer that is one of four: below 0.035 x
sqrt(4) x sqrt(2) = 0.1 with the layers behind it."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rope,q4,bound", [(True, False, 2.3e-2), (False, True, 0.1), (True, True, 0.1)])
@pytest.mark.parametrize("lens,parts", [((300, 1, 77, 130), 3), ((5, 900), 4)])
def test_steps_equal_one_step(lens, parts, rope, q4, bound):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_delta_rule_40_gb300 import hybrid_example
    assert hybrid_example.main(lens, parts, rope=rope, q4=q4) < bound
