"""Layouts that the binding of the gated-delta and beam entries refuses before the library is called (CPU)."""
import pytest
import torch

from linear_rnn_sequence_rwkv_b200 import wkv7


def _tokens(B, T, H=4, Hk=2, N=64):
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    return {"q": z(B, T, Hk, N), "k": z(B, T, Hk, N), "v": z(B, T, H, N), "g": z(B, T, H), "beta": z(B, T, H)}


@pytest.mark.parametrize("name", ["q", "k", "v"])
@pytest.mark.parametrize("B,T,kept", [(2, 3, (1, 1)), (2, 3, (1, 3)), (1, 3, (1, 1)), (3, 1, (1, 1)), (2, 3, (2, 1))])
def test_rows_expanded_over_tokens_or_sequences(name, B, T, kept):
    """One stored row that stands for several has a stride of 0, which the library would take for dense rows."""
    d = _tokens(B, T)
    d[name] = d[name][:kept[0], :kept[1]].expand(d[name].shape)
    dy, S = torch.zeros_like(d["v"]), None
    with pytest.raises(ValueError, match=f"{name}: its rows"):
        wkv7.delta_forward(*d.values())
    with pytest.raises(ValueError, match=f"{name}: its rows"):
        wkv7.delta_backward(*d.values(), dy, S)


@pytest.mark.parametrize("name", ["q", "k", "v"])
def test_rows_expanded_in_a_step_and_when_packed(name):
    d = {n: x[0] for n, x in _tokens(1, 5).items()}
    d[name] = d[name][:1].expand(d[name].shape)
    with pytest.raises(ValueError, match=f"{name}: its rows"):
        wkv7.delta_step(*d.values(), torch.zeros(5, 4, 64, 64))
    with pytest.raises(ValueError, match=f"{name}: its rows"):
        wkv7.delta_forward(*d.values(), cu_seqlens=torch.tensor([0, 5], dtype=torch.int32))


def test_rows_that_overlap():
    x = torch.zeros(4096, dtype=torch.bfloat16)
    v = x.as_strided((1, 6, 4, 64), (256, 64, 64, 1))
    with pytest.raises(ValueError, match="v: its rows"):
        wkv7._row_stride("v", v, v.shape, v.dtype, v.device)


def test_one_row_has_no_stride():
    x = torch.zeros(1, 1, 2, 64)
    assert wkv7._row_stride("q", x.expand(1, 1, 2, 64), (1, 1, 2, 64), torch.float32, x.device) == 0


@pytest.mark.parametrize("B,K,kept", [(1, 4, (1, 1)), (3, 4, (1, 1)), (3, 1, (1, 1)), (3, 4, (3, 1)), (3, 4, (1, 4))])
def test_logits_expanded_over_beams_or_requests(B, K, kept):
    """As in a search's first step, where every beam of a request has the prompt's logits."""
    x = torch.zeros(*kept, 50, dtype=torch.bfloat16).expand(B, K, 50)
    with pytest.raises(ValueError, match="logits: its rows"):
        wkv7.beam_select(x, torch.zeros(B, K), 2)


def test_logits_whose_rows_overlap():
    x = torch.zeros(200).as_strided((2, 3, 50), (30, 10, 1))
    with pytest.raises(ValueError, match="logits: its rows"):
        wkv7.beam_select(x, torch.zeros(2, 3), 2)
    with pytest.raises(ValueError, match="logits: its rows"):
        wkv7.beam_select(torch.zeros(1, 1, 1).expand(2, 3, 1), torch.zeros(2, 3), 2)


@pytest.mark.parametrize("scale", [0, 0.0, -0.0, 1e-60])
def test_a_scale_of_zero(scale):
    """The library reads 0 as its default, 1 / sqrt(N): a caller's own zero is not that."""
    d = _tokens(1, 3)
    with pytest.raises(ValueError, match="scale"):
        wkv7.delta_forward(*d.values(), scale=scale)
    with pytest.raises(ValueError, match="scale"):
        wkv7.delta_backward(*d.values(), torch.zeros_like(d["v"]), scale=scale)
    with pytest.raises(ValueError, match="scale"):
        wkv7.delta_step(*(x[0] for x in d.values()), torch.zeros(3, 4, 64, 64), scale=scale)


def test_a_workspace_with_gaps():
    """Its elements' bytes would count as dense, and what lies between them be overwritten."""
    cpu = torch.device("cpu")
    with pytest.raises(ValueError, match="workspace"):
        wkv7._workspace(torch.zeros(100, dtype=torch.uint8)[::2], 40, cpu)
    with pytest.raises(ValueError, match="workspace"):
        wkv7._workspace(torch.zeros(1).expand(100), 40, cpu)
    own = torch.zeros(20)
    assert wkv7._workspace(own, 80, cpu)[0] is own and wkv7._workspace(own, 80, cpu)[1] == 80
    new, size = wkv7._workspace(own, 81, cpu)
    assert new is not own and size == 81 and wkv7._workspace(None, 0, cpu) == (None, 0)
