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


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 3, 7, 8, 9, 15, 16, 17, 31, 257, 2049, 50277])
@pytest.mark.parametrize("off", [1, 2, 3, 4, 5, 6, 7])
def test_logits_that_start_anywhere(cuda_device, off, V, dt):
    """Rows cut from the middle of a buffer, which holds other things right before and behind them."""
    B, K, M = 2, 3, 9
    g = torch.Generator().manual_seed(off + V)
    x, s = (3 * torch.randn(B, K, V, generator=g)).to(DT[dt]), torch.randn(B, K, generator=g)
    held = torch.full((off + B * K * V + 16,), float("inf"), dtype=DT[dt], device=cuda_device)
    held[off + B * K * V:] = float("nan")
    view = held[off:off + B * K * V].view(B, K, V)
    view.copy_(x)
    got = wkv7.beam_select(view, s.to(cuda_device), M)
    ref = wkv7.beam_select(x.to(cuda_device), s.to(cuda_device), M)
    for a, b in zip(got, ref):
        assert torch.equal(a, b)
    want = delta.beam_select(x.double().numpy(), s.numpy(), M)
    assert np.array_equal(got[1].cpu().numpy(), want[1]) and np.array_equal(got[2].cpu().numpy(), want[2])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_logits_of_the_last_position(cuda_device, dt):
    """[B, K] prompts of T tokens each, an odd vocabulary: the last position's rows are a strided view."""
    B, K, T, V, M = 2, 4, 3, 4099, 8
    g = torch.Generator().manual_seed(5)
    x, s = (3 * torch.randn(B, K, T, V, generator=g)).to(DT[dt]), torch.randn(B, K, generator=g)
    xd = x.to(cuda_device)
    got = wkv7.beam_select(xd[:, :, -1], s.to(cuda_device), M)
    want = delta.beam_select(x[:, :, -1].double().numpy(), s.numpy(), M)
    assert np.array_equal(got[1].cpu().numpy(), want[1]) and np.array_equal(got[2].cpu().numpy(), want[2])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_beams_at_the_lowest_score_offer_their_tokens_by_logit(cuda_device, dt):
    """The tokens of one beam come in the order of their logits, whatever its score leaves of their differences."""
    g = torch.Generator().manual_seed(6)
    x = (3 * torch.randn(1, 3, 501, generator=g)).to(DT[dt])
    low = torch.finfo(torch.float32).min
    got = wkv7.beam_select(x.to(cuda_device), torch.full((1, 3), low, device=cuda_device), 7)
    order = torch.sort(x[0, 0].float(), descending=True, stable=True).indices[:7]
    assert got[1].tolist() == [[0] * 7] and got[2].cpu().tolist() == [order.tolist()]
    assert bool(torch.all(got[0] == low))
    s = torch.tensor([[low, -3.0, low]])
    got = wkv7.beam_select(x.to(cuda_device), s.to(cuda_device), 7)
    assert got[1].tolist() == [[1] * 7]
