"""The example's beam search with one set of states that beam_reorder moves."""
import importlib.util
import os

import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("eos", [None, 5])
def test_moved_states_decode_as_two_sets(eos):
    """Both ways compute each beam's step from the same state: the same tokens and scores, bit for bit."""
    spec = importlib.util.spec_from_file_location("causal_lm", os.path.join(ROOT, "examples", "causal_lm.py"))
    lm = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(lm)
    say("case example moved states %s" % eos)
    p = lm.init(seed=4)
    t = lm.progressions(5, 16, torch.Generator().manual_seed(6))
    lengths = torch.tensor([3, 16, 1, 7, 12], dtype=torch.int32).cuda()
    for beams in (1, 4, 7):
        a = lm.beam_search(p, t, lengths, beams, 9, eos=eos)
        b = lm.beam_search(p, t, lengths, beams, 9, eos=eos, move=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), beams
        assert len({tuple(v) for v in a[0].reshape(-1, 9).tolist()}) > beams
