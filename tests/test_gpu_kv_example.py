"""The example layer (examples/decode_layer.py): quantised projections, cache and attention together; the last
step's attention against the dense one on the cache read back.  Both round to fp16 (the read-back, the
attention's weights and its output, 2^-11 each): 4e-3 in the 2-norm is eight such roundings."""
import pytest

from tests.gpu_common import say, torch_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prompt,answers,steps,nbits", [(700, 16, 40, 4), (65, 3, 70, 8), (1, 1, 1, 4)])
def test_decode_layer(prompt, answers, steps, nbits):
    torch_dev()
    from examples import decode_layer
    say("decode layer", prompt, answers, steps, nbits)
    assert decode_layer.main(prompt, answers, steps, nbits) <= 4e-3
