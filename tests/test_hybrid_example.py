"""GPU test of the hybrid decoder that runs the page plan, the cache write and both attention calls next to
the KDA layers: the same prompts in one step and in chunks give the same last logits.

Tolerance: both decoders round the same activations to bf16 (2^-8 each) at different places of two paths
(whole prompt and paged; one chunking of the KDA state and another).  A handful of independent roundings a
layer over four layers stays below sqrt(4 x 8) 2^-8 = 2.2e-2 relative."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,parts", [((300, 1, 77, 130), 3), ((64, 65), 1), ((5, 900), 4)])
def test_steps_equal_one_step(lens, parts):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_delta_rule_40_gb300 import hybrid_example
    assert hybrid_example.main(lens, parts) < 2.2e-2
