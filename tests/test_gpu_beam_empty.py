"""kda_state_reorder where a parent's slot holds nothing: its first child keeps that slot, the others take slots whose
contents stay as they were (there is no state to copy), and a step of a search whose empty beams have scores of
-infinity never has such a parent."""

import pytest
import torch

from gated_delta_rule_10_amd import beam

pytestmark = pytest.mark.gpu


def test_children_of_a_beam_that_holds_nothing():
    states = torch.arange(6 * 64, dtype=torch.float32, device="cuda").view(1, 6, 64)
    before = states.clone()
    slots = torch.tensor([[-1, 3, 5, 0]], dtype=torch.int32, device="cuda")
    out = beam.kda_state_reorder(states, slots, torch.tensor([[0, 0, 3, 3]], dtype=torch.int32, device="cuda"))
    assert out.tolist() == [[-1, 3, 0, 5]]
    assert torch.equal(states[0, [0, 1, 2, 3, 4]], before[0, [0, 1, 2, 3, 4]]) and torch.equal(states[0, 5], before[0, 0])


def test_a_search_does_not_go_on_from_such_beams():
    """Three of four beams hold nothing and have scores of -infinity: all four go on from the one."""
    logits = torch.randn((2, 4, 500), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    scores = torch.full((2, 4), -float("inf"), device="cuda")
    scores[0, 2] = scores[1, 0] = -1.5
    _, parent, _ = beam.kda_beam_select(logits, scores, 4)
    assert parent.tolist() == [[2] * 4, [0] * 4]
