"""The gated delta rule at the edges of its contract."""
import numpy as np
import pytest
import torch

from linear_rnn_sequence_rwkv_b200 import wkv7
from oracle import delta
from tests.delta_util import DT, Y_TOL, make, state
from tests.parity_util import slice_rel_err

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
# ---- states that grow -----------------------------------------------------------------------------

# fp32: the exponent's own rounding, 81 * 2^-24 = 5e-6 relative, in each of at most four decays behind an output, above
# the 1e-5 that fp32 is held to elsewhere. bf16: as elsewhere.
GROW_TOL = {"bf16": Y_TOL["bf16"], "f32": 3e-5}


def grown(got, ref, dt):
    """Token by token: the error against the largest output so far (outputs grow by orders of magnitude)."""
    got, ref = got.double().cpu().numpy(), np.asarray(ref)
    top = np.maximum.accumulate(np.abs(ref).max(-1), axis=1)
    return np.all(np.abs(got - ref).max(-1) <= GROW_TOL[dt] * top + 1e-37)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("gates", [[5.0] * 15 + [-75.0], [2.0] * 37 + [-74.0], [-100.0] + [4.0] * 18 + [-72.0]])
def test_states_that_grow(cuda_device, gates, N, dt):
    """Positive log decays, by less than e^80 within 32 tokens."""
    T = 100
    d = make((1, T), 2, 2, N, dt, seed=73)
    d["g"][:] = torch.tensor((gates * T)[:T]).to(DT[dt])[None, :, None]
    d["v"] *= 1e-12
    y, S = wkv7.delta_forward(*to(d, cuda_device).values(), qk_norm=True)
    yr, Sr = delta.delta_recurrence(*d.values(), qk_norm=True)
    assert bool(torch.isfinite(y).all()) and grown(y, yr, dt)
    assert np.abs(S.double().cpu().numpy() - Sr).max() <= GROW_TOL["f32"] * np.abs(Sr).max()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("gates,over", [([3.0] * 32, 26), ([-1.0] * 5 + [-100.0] + [5.0] * 26, 22),
                                        ([0.0] * 32 + [-110.0] + [8.0] * 11 + [-60.0] * 20, 43),
                                        ([-1.0] * 9 + [85.0] + [-85.0] * 22, 9), ([-1.0] * 70 + [81.0], 70)])
@pytest.mark.parametrize("first_state", [False, True])
def test_states_that_grow_too_much(cuda_device, first_state, gates, over, N, dt):
    """By more than e^80 within a block of 32 tokens: not finite from that token on, whatever the state holds; what
    comes before, and the other heads, are as they were."""
    T = 130
    d = make((1, T), 4, 2, N, dt, seed=74)
    d["v"] *= 1e-12
    S0 = 1e-12 * state(1, 4, N, 5).to(cuda_device) if first_state else None
    ref = wkv7.delta_forward(*to(d, cuda_device).values(), S0, qk_norm=True)
    d["g"][:, :, 1] = torch.tensor((gates + [-1.0] * T)[:T]).to(DT[dt])[None]
    y, S = wkv7.delta_forward(*to(d, cuda_device).values(), S0, qk_norm=True)
    other = [0, 2, 3]
    assert torch.equal(y[:, :, other], ref[0][:, :, other]) and torch.equal(S[:, other], ref[1][:, other])
    one = {n: x[:, :over, 0 if n in "qk" else 1][:, :, None] for n, x in d.items()}
    yr, _ = delta.delta_recurrence(*one.values(), None if S0 is None else S0[:, 1:2].cpu(), qk_norm=True)
    assert grown(y[:, :over, 1:2], yr, dt)
    assert not bool(torch.isfinite(y[:, over:, 1]).any()) and not bool(torch.isfinite(S[:, 1]).any())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("gates", [[1.0] * 30 + [-30.0], [-50.0] + [2.0] * 20 + [-40.0]])
def test_gradients_of_states_that_grow(cuda_device, gates, N, dt):
    """By less than e^80 within 64 tokens. fp32: the exponents' rounding, 50 * 2^-24 = 3e-6 in each of at most four decays
    behind a gradient, above the 2e-5 that fp32 gradients are held to: 4e-5 of a head's largest. bf16: as elsewhere."""
    T = 130
    d = make((1, T), 2, 1, N, dt, seed=77)
    d["g"][:] = torch.tensor((gates * T)[:T]).to(DT[dt])[None, :, None]
    d["v"] *= 1e-6
    g = torch.Generator().manual_seed(78)
    dy, dS = torch.randn(1, T, 2, N, generator=g).to(DT[dt]), 0.1 * torch.randn(1, 2, N, N, generator=g)
    got = wkv7.delta_backward(*to(d, cuda_device).values(), dy.to(cuda_device), None, dS.to(cuda_device), qk_norm=True)
    ref = delta.delta_backward(*d.values(), None, dy, dS, qk_norm=True)
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert slice_rel_err(got[n], ref[n], (0, 2)) <= (Y_TOL["bf16"] if dt == "bf16" else 4e-5), n
    assert slice_rel_err(got["dS0"], ref["dS0"], (0, 1)) <= 4e-5
# ---- keys and queries whose squares leave fp32 -------------------------------------------------------

@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("t", [0, 45, 69])
def test_lengths_beyond_fp32_are_not_finite(cuda_device, t, N, dt):
    """With qk_norm a key or query whose sum of squares overflows fp32 counts as one that is not finite."""
    d = make((1, 70), 4, 2, N, dt, seed=75)
    ref, S_ref = wkv7.delta_forward(*to(d, cuda_device).values(), qk_norm=True)
    for name in "kq":
        x = {n: v.clone() for n, v in d.items()}
        x[name][0, t, 1, 5] = 1e20
        y, S = wkv7.delta_forward(*to(x, cuda_device).values(), qk_norm=True)
        assert torch.equal(y[:, :, :2], ref[:, :, :2]) and torch.equal(S[:, :2], S_ref[:, :2])
        tol = Y_TOL[dt] * float(ref.abs().max())
        assert t == 0 or float((y[:, :t, 2:] - ref[:, :t, 2:]).abs().max()) <= tol
        if name == "k":
            assert not bool(torch.isfinite(y[:, t:, 2:]).any()) and not bool(torch.isfinite(S[:, 2:]).any())
        else:
            assert not bool(torch.isfinite(y[:, t, 2:]).any()) and torch.equal(S, S_ref)
            assert t == 69 or float((y[:, t + 1:, 2:] - ref[:, t + 1:, 2:]).abs().max()) <= tol
        one = {n: v[:, t].contiguous().to(cuda_device) for n, v in x.items()}
        pool = state(1, 4, N, 6).to(cuda_device)
        before = pool.clone()
        y1 = wkv7.delta_step(*one.values(), pool, qk_norm=True)
        assert bool(torch.isfinite(y1[:, :2]).all()) and bool(torch.isfinite(pool[:, :2]).all())
        assert not bool(torch.isfinite(y1[:, 2:]).any())
        assert bool(torch.isfinite(pool[:, 2:]).any()) == (name == "q")
        assert not torch.equal(pool[:, :2], before[:, :2])
        dy = torch.ones_like(x["v"]).to(cuda_device)
        g = wkv7.delta_backward(*to(x, cuda_device).values(), dy, qk_norm=True)
        assert not bool(torch.isfinite(g["d" + name][0, t, 1]).any())
# ---- fp32 beyond bf16's range -------------------------------------------------------------------------

@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("t", [0, 45, 69])
@pytest.mark.parametrize("value", [torch.finfo(torch.float32).min, 3.4e38])
def test_values_beyond_the_range_of_bf16(cuda_device, value, t, N):
    """Operands are split into bf16 terms, the largest of which is 3.39e38: an fp32 value above it counts as infinite,
    and like one reaches its own channel from its token on and nothing else."""
    d = make((1, 70), 2, 2, N, "f32", seed=76)
    ref, S_ref = wkv7.delta_forward(*to(d, cuda_device).values(), qk_norm=True)
    d["v"][0, t, 1, 7] = value
    y, S = wkv7.delta_forward(*to(d, cuda_device).values(), qk_norm=True)
    rest = [i for i in range(N) if i != 7]
    tol = Y_TOL["f32"] * float(ref.abs().max())
    assert torch.equal(y[:, :, 0], ref[:, :, 0])
    assert float((y[..., rest] - ref[..., rest]).abs().max()) <= tol
    assert t == 0 or float((y[:, :t] - ref[:, :t]).abs().max()) <= tol
    assert not bool(torch.isfinite(y[0, t:, 1, 7]).any()) and not bool(torch.isfinite(S[0, 1, 7]).any())
    assert bool(torch.isfinite(S[0, 1, rest]).all())
