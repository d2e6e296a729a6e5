"""The gated delta rule at the edges of its contract."""
import numpy as np
import pytest
import torch

from linear_rnn_sequence_rwkv_b200 import wkv7
from oracle import delta
from tests.delta_util import DT, TOK, Y_TOL, make, state

pytestmark = pytest.mark.gpu


def to(d, dev):
    return {n: x.to(dev) for n, x in d.items()}


# ---- dg where the state cannot matter ------------------------------------------------------------

@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("with_state", [False, True])
def test_dg_is_zero_where_the_state_is_forgotten(cuda_device, with_state, N, dt):
    """exp(g) is 0 in fp32: S_t does not depend on g, to the last bit. Nor does it at a first token without S0."""
    B, T, H = 2, 150, 3
    d = make((B, T), H, 1, N, dt, seed=71)
    at = [20, 31, 32, 63, 64, 100, 149]
    for i, t in enumerate(at):
        d["g"][:, t] = (float("-inf"), -104.5, -1e30)[i % 3]
    S0 = state(B, H, N, 1).to(cuda_device) if with_state else None
    dy = torch.randn(B, T, H, N, generator=torch.Generator().manual_seed(2)).to(DT[dt]).to(cuda_device)
    dS = state(B, H, N, 3).to(cuda_device)
    dg = wkv7.delta_backward(*to(d, cuda_device).values(), dy, S0, dS, qk_norm=True)["dg"]
    assert bool(torch.all(dg[:, at] == 0))
    assert bool(torch.all(dg[:, 0] == 0)) == (not with_state)
    rest = [t for t in range(1, T) if t not in at]
    assert float((dg[:, rest] != 0).float().mean()) > 0.9


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_dg_is_zero_at_the_first_tokens_of_packed_sequences(cuda_device, dt):
    lens, H, N = [3, 0, 64, 1, 130, 65], 4, 64
    cu = [0, *np.cumsum(lens).tolist()]
    d = make((cu[-1],), H, 2, N, dt, seed=72)
    dy = torch.randn(cu[-1], H, N, generator=torch.Generator().manual_seed(3)).to(DT[dt]).to(cuda_device)
    got = wkv7.delta_backward(*to(d, cuda_device).values(), dy, qk_norm=True,
                              cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=cuda_device))
    first = [a for a, n in zip(cu, lens) if n]
    assert bool(torch.all(got["dg"][first] == 0))
    assert bool(torch.all(got["dg"][[a + 1 for a, n in zip(cu, lens) if n > 1]] != 0))
