"""The drafting example (examples/draft_layer.py): plan, rotated write, attention for trees and accepted drafts together against decoding the
accepted tokens one by one.  Both attend over the same bytes, in streamed rows; each rounds its weights, code * step and the output to
fp16 (2^-11 each, 1e-3 in the 2-norm at most where the errors do not cancel): 2e-3 between the two.  The caches stand for the same values
bit for bit."""
import pytest

from tests.gpu_common import say, torch_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("answers,drafts,steps,nbits", [(8, 16, 6, 4), (3, 26, 4, 8), (1, 1, 3, 4), (5, 64, 2, 4)])
def test_draft_layer(answers, drafts, steps, nbits):
    torch_dev()
    from examples import draft_layer
    say("draft layer", answers, drafts, steps, nbits)
    worst, equal = draft_layer.main(answers, drafts, steps, nbits=nbits)
    assert equal and worst <= 2e-3
