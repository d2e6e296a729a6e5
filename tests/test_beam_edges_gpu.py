"""Beam selection at the edges of its contract: signed zeros, logits that start anywhere, beams at the lowest score."""
import numpy as np
import pytest
import torch

from linear_rnn_sequence_rwkv_b200 import wkv7
from oracle import delta
from tests.delta_util import DT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_scores_of_minus_zero_tie_with_zero(cuda_device, dt):
    """Finished beams keep their own score: -0 and 0 are one score, and the lowest beam comes first."""
    s = torch.tensor([[-0.0, 0.0, -0.0, -1.0], [0.0, -0.0, 0.0, -0.0]])
    f = torch.ones(2, 4, dtype=torch.bool)
    x = torch.zeros(2, 4, 33, dtype=DT[dt])
    got = wkv7.beam_select(x.to(cuda_device), s.to(cuda_device), 4, finished=f.to(cuda_device), eos=3)
    assert got[1].tolist() == [[0, 1, 2, 3], [0, 1, 2, 3]]
    assert torch.equal(got[0].cpu(), torch.tensor([[0.0, 0.0, 0.0, -1.0], [0.0, 0.0, 0.0, 0.0]]))
    # beside a live beam whose only token has probability 1
    x = torch.zeros(1, 3, 1, dtype=DT[dt])
    s, f = torch.tensor([[-0.0, 0.0, -0.0]]), torch.tensor([[True, False, True]])
    got = wkv7.beam_select(x.to(cuda_device), s.to(cuda_device), 3, finished=f.to(cuda_device), eos=0)
    assert got[1].tolist() == [[0, 1, 2]]
