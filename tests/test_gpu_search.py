"""The example's search at its smallest: one token, one beam, and both."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import state_space_lm as lm  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mixer", ["gated", "selective"])
@pytest.mark.parametrize("beams", [1, 3])
def test_one_token(mixer, beams):
    torch.manual_seed(7)
    model = lm.Model(9, model=16, inner=24, layers=1, mixer=mixer).cuda()
    prompt = torch.randint(0, 9, (2, 5), device="cuda")
    text, scores = lm.search(model, prompt, 1, beams)
    with torch.no_grad():
        want, tokens = torch.log_softmax(model(prompt)[0][:, -1].double(), -1).topk(beams)
    assert text.shape == (2, beams, 1) and torch.equal(text[..., 0].long(), tokens)
    # one rounding to float32, 2^-24, and as much again for 64-bit sums in another order
    assert bool(((scores.double() - want).abs() <= 2.0 ** -23 * want.abs()).all())


def test_one_beam_is_greedy():
    torch.manual_seed(8)
    model = lm.Model(11, model=16, inner=24, layers=2, mixer="gated").cuda()
    prompt = torch.randint(0, 11, (3, 6), device="cuda")
    text, _ = lm.search(model, prompt, 7, 1)
    tokens, _ = lm.answer(model, prompt, 7)
    assert torch.equal(text[:, 0].long(), tokens)
