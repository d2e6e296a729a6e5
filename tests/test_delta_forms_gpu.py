"""Every form that the launches of the gated delta rule choose between, by the number of heads, against the oracle.

bf16 at N = 64 has two forward kernels (up to 74 heads over all sequences, and above) and two pairs of sweeps in the
backward (up to 37, and above); the sweeps run in one launch up to 74 blocks and in turn above. The value heads of a
key head are divided where chunks and key heads leave SMs idle. The bounds are those of the other tests: one rounding of
the result and of two operands for bf16, 1e-5 (gradients 2e-5) for fp32.
"""
import numpy as np
import pytest
import torch

from linear_rnn_sequence_rwkv_b200 import wkv7
from oracle import delta
from tests.delta_util import DT, S_TOL, TOK, Y_TOL, make, s_err, state, y_err
from tests.parity_util import slice_rel_err

pytestmark = pytest.mark.gpu
G_TOL = {"bf16": 3 * 2.0 ** -8, "f32": 2e-5}
NAMES = ("dq", "dk", "dv", "dg", "dbeta")


def to(d, dev):
    return {n: x.to(dev) for n, x in d.items()}


def check(got, ref, dt, floor=None):
    """floor: what dg and dbeta may be off by besides, per sequence and head."""
    for n in NAMES:
        if ref[n].size and floor is not None and n in floor:
            off = np.abs(got[n].double().cpu().numpy() - ref[n]).max(1)
            assert np.all(off <= G_TOL[dt] * np.abs(ref[n]).max(1) + floor[n]), n
        elif ref[n].size:
            assert slice_rel_err(got[n], ref[n], (0, 2)) <= G_TOL[dt], n
    assert slice_rel_err(got["dS0"], ref["dS0"], (0, 1)) <= G_TOL["f32"]


def floor_of_one_token(d, dy, S0, dS):
    """With one token a slice of dg or dbeta is a single number, and nothing bounds it from below: dg = <P, dP> with
    P = exp(g) S0 cancels N^2 products, dbeta = <du, e> N of them. A sum is off by the roundings on the way from a product
    to the result, relative to the sum of the products' sizes, which is at most |P| |dP| and |du| |e| (Cauchy-Schwarz).
    On the way: operands in three bf16 terms (2 x 2^-24), the state's products N / 16 accumulations that cut
    (2^-23 each, N <= 128: 16 x 2^-24), at most 8 x 4 fused steps per thread, 5 + 4 + 5 levels of adding up: below
    2^6 x 2^-24 = 2^-18. With unit k and q of length scale: |du| <= |dS| + scale |dy|, |dP| <= 2 |du| (beta <= 1),
    |e| <= |v| + |P|."""
    B, _, H, N = d["v"].shape
    size = lambda x: np.sqrt((x.double().numpy() ** 2).reshape(B, H, -1).sum(-1))  # noqa: E731
    P = np.exp(d["g"][:, 0].double().numpy()) * size(S0)
    du = size(dS) + N ** -0.5 * size(dy[:, 0])
    return {"dg": 2.0 ** -18 * P * 2 * du, "dbeta": 2.0 ** -18 * du * (size(d["v"][:, 0]) + P)}


@pytest.mark.parametrize("B,H,Hk", [(2, 37, 37), (1, 74, 2), (3, 25, 5), (1, 75, 75), (5, 30, 6), (8, 40, 8)])
@pytest.mark.parametrize("T", [31, 200, 333])
def test_forward_by_heads(cuda_device, T, B, H, Hk):
    d = make((B, T), H, Hk, 64, "bf16", seed=B * H + T)
    S0 = state(B, H, 64, T)
    y, S = wkv7.delta_forward(*to(d, cuda_device).values(), S0.to(cuda_device), qk_norm=True)
    yr, Sr = delta.delta_recurrence(*d.values(), S0, qk_norm=True)
    assert y_err(y, yr) <= Y_TOL["bf16"] and s_err(S, Sr) <= S_TOL


@pytest.mark.parametrize("H", [12, 15, 16, 40])
def test_forward_packed_by_heads(cuda_device, H):
    """60 to 200 heads over five sequences, an empty one and one of a single token among them; rows behind them stay."""
    lens, tail, Hk, N = [270, 0, 1, 170, 64], 9, H // (4 if H % 4 == 0 else 5), 64
    cu = [0, *np.cumsum(lens).tolist()]
    d = make((cu[-1] + tail,), H, Hk, N, "bf16", seed=H)
    d["v"][cu[-1]:] = float("nan")
    S0 = state(len(lens), H, N, 3)
    y = torch.full_like(d["v"], 5.0).to(cuda_device)
    _, S = wkv7.delta_forward(*to(d, cuda_device).values(), S0.to(cuda_device), qk_norm=True, y=y,
                              cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=cuda_device))
    for s, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        yr, Sr = delta.delta_recurrence(*(d[n][a:b][None] for n in TOK), S0[s:s + 1], qk_norm=True)
        assert s_err(S[s:s + 1], Sr) <= S_TOL and (a == b or y_err(y[a:b][None], yr) <= Y_TOL["bf16"])
    assert torch.all(y[cu[-1]:] == 5.0)


def test_forward_strided_rows_with_many_heads(cuda_device):
    H, Hk, N, B, T = 40, 8, 64, 3, 250
    d = make((B, T), H, Hk, N, "bf16", seed=16)
    wide = torch.cat([d["q"].flatten(2), d["k"].flatten(2), d["v"].flatten(2)], dim=-1).to(cuda_device)
    q, k, v = wide.split([Hk * N, Hk * N, H * N], dim=-1)
    y, S = wkv7.delta_forward(q.unflatten(-1, (Hk, N)), k.unflatten(-1, (Hk, N)), v.unflatten(-1, (H, N)),
                              d["g"].to(cuda_device), d["beta"].to(cuda_device), qk_norm=True)
    y2, S2 = wkv7.delta_forward(*to(d, cuda_device).values(), qk_norm=True)
    assert torch.equal(y, y2) and torch.equal(S, S2)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("t", [0, 45, 199])
def test_forward_inputs_that_are_not_finite_with_many_heads(cuda_device, t, bad):
    B, T, H, Hk, N = 2, 200, 40, 20, 64
    d = make((B, T), H, Hk, N, "bf16", seed=17)
    ref, S_ref = wkv7.delta_forward(*to(d, cuda_device).values(), qk_norm=True)
    for name, heads in (("q", [2, 3]), ("k", [2, 3]), ("v", [2]), ("g", [2]), ("beta", [2])):
        x = {n: v.clone() for n, v in d.items()}
        x[name][(1, t, 1, 7) if name in "qk" else (1, t, 2, 7) if name == "v" else (1, t, 2)] = bad
        y, S = wkv7.delta_forward(*to(x, cuda_device).values(), qk_norm=True)
        other = [h for h in range(H) if h not in heads]
        assert torch.equal(y[0], ref[0]) and torch.equal(S[0], S_ref[0]), name
        assert torch.equal(y[1][:, other], ref[1][:, other]) and torch.equal(S[1, other], S_ref[1, other]), name
        mine, was = y[1][:, heads], ref[1][:, heads]
        tol = Y_TOL["bf16"] * float(was.abs().max())
        assert t == 0 or float((mine[:t] - was[:t]).abs().max()) <= tol, name
        if name == "v":
            assert not torch.isfinite(mine[t:, :, 7]).any() and not torch.isfinite(S[1, 2, 7]).any()
            keep = [i for i in range(N) if i != 7]
            assert float((mine[..., keep] - was[..., keep]).abs().max()) <= tol
        elif name == "q":
            assert not torch.isfinite(mine[t]).any() and torch.equal(S[1], S_ref[1])
        else:
            assert not torch.isfinite(mine[t:]).any() and not torch.isfinite(S[1, heads]).any()


@pytest.mark.parametrize("dt,N,B,H,Hk", [("bf16", 64, 1, 37, 37), ("bf16", 64, 2, 19, 19), ("bf16", 64, 2, 37, 1),
                                         ("bf16", 64, 3, 25, 5), ("bf16", 64, 4, 40, 10), ("f32", 64, 2, 37, 37),
                                         ("f32", 64, 3, 25, 5), ("f32", 64, 5, 20, 20), ("bf16", 128, 3, 26, 13),
                                         ("f32", 128, 2, 20, 4)])
@pytest.mark.parametrize("T", [1, 33, 200])
def test_backward_by_heads(cuda_device, T, dt, N, B, H, Hk):
    d = make((B, T), H, Hk, N, dt, seed=B * H + T)
    g = torch.Generator().manual_seed(T)
    dy, dS = torch.randn(B, T, H, N, generator=g).to(DT[dt]), 0.1 * torch.randn(B, H, N, N, generator=g)
    S0 = state(B, H, N, T)
    got = wkv7.delta_backward(*to(d, cuda_device).values(), dy.to(cuda_device), S0.to(cuda_device), dS.to(cuda_device), qk_norm=True)
    check(got, delta.delta_backward(*d.values(), S0, dy, dS, qk_norm=True), dt,
          floor_of_one_token(d, dy, S0, dS) if T == 1 else None)


@pytest.mark.parametrize("dt,H,Hk", [("bf16", 7, 7), ("bf16", 8, 2), ("bf16", 16, 16), ("f32", 16, 4)])
def test_backward_packed_by_heads(cuda_device, dt, H, Hk):
    lens, N = [190, 0, 1, 130, 64], 64
    cu = [0, *np.cumsum(lens).tolist()]
    d = make((cu[-1],), H, Hk, N, dt, seed=H)
    g = torch.Generator().manual_seed(H)
    dy, dS = torch.randn(cu[-1], H, N, generator=g).to(DT[dt]), 0.1 * torch.randn(len(lens), H, N, N, generator=g)
    S0 = state(len(lens), H, N, 3)
    got = wkv7.delta_backward(*to(d, cuda_device).values(), dy.to(cuda_device), S0.to(cuda_device), dS.to(cuda_device),
                              qk_norm=True, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=cuda_device))
    for s, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        ref = delta.delta_backward(*(d[n][a:b][None] for n in TOK), S0[s:s + 1], dy[a:b][None], dS[s:s + 1], qk_norm=True)
        check({**{n: got[n][a:b][None] for n in NAMES}, "dS0": got["dS0"][s:s + 1]}, ref, dt)


def test_backward_rows_past_32_bit_offsets(cuda_device):
    """2^31 elements of v, and of what is kept per row, lie before the second sequence."""
    H, N, n = 64, 64, 40
    rows = 2 ** 31 // (H * N) + 24 + n
    if torch.cuda.mem_get_info()[0] < 90e9:
        pytest.skip("needs 90 GB")
    d = make((1, n), H, 1, N, "bf16", seed=23)
    dy1 = torch.randn(1, n, H, N, generator=torch.Generator().manual_seed(24)).bfloat16()
    new = lambda *s: torch.zeros(rows, *s, device=cuda_device, dtype=torch.bfloat16)  # noqa: E731
    x = {"q": new(1, N), "k": new(1, N), "v": new(H, N), "g": new(H) - 1.0, "beta": new(H)}
    dy = new(H, N)
    for name in TOK:
        x[name][rows - n:] = d[name][0].to(cuda_device)
    dy[rows - n:] = dy1[0].to(cuda_device)
    got = wkv7.delta_backward(*x.values(), dy, qk_norm=True,
                              cu_seqlens=torch.tensor([0, rows - n, rows], dtype=torch.int32, device=cuda_device))
    ref = delta.delta_backward(*d.values(), None, dy1, None, qk_norm=True)
    check({**{m: got[m][rows - n:][None] for m in NAMES}, "dS0": got["dS0"][1:]}, ref, "bf16")
    assert all(bool(torch.all(got[m][:rows - n] == 0)) for m in ("dv", "dq", "dk", "dbeta"))
