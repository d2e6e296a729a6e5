"""The gated delta rule's gradients on the GPU against the fp64 oracle's chain rule and differences.

Bounds (max error over a slice relative to the slice's largest reference value; a slice is a
sequence and head). fp32: 2e-5, twice the forward's bound, since a gradient passes through the
forward's sums and the reverse ones. bf16 outputs: the result's own rounding (2^-8 of the value) and
one rounding of an operand in each of at most four sums that make it up (the states' and their gradients'
2^-8, with signs that vary): 3 * 2^-8 as for y. The state's gradient is fp32 throughout: 2e-5. dg and
dbeta are single numbers per token, each a sum over N channels whose operands are rounded so: the
same bound against the slice's largest.
"""
import numpy as np
import pytest
import torch

from linear_rnn_sequence_rwkv_b200 import wkv7
from oracle import delta
from tests.delta_util import TOK, make, state
from tests.parity_util import slice_rel_err

pytestmark = pytest.mark.gpu
TOL = {"bf16": 3 * 2.0 ** -8, "f32": 2e-5}
S_TOL = 2e-5
NAMES = ("dq", "dk", "dv", "dg", "dbeta")


def to(d, dev):
    return {n: x.to(dev) for n, x in d.items()}


def extra(lead, B, H, N, dt, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*lead, H, N, generator=g).to(torch.bfloat16 if dt == "bf16" else torch.float32),
            0.1 * torch.randn(B, H, N, N, generator=g))


def check(got, ref, dt, names=NAMES):
    for n in names:
        if ref[n].size:
            assert slice_rel_err(got[n], ref[n], (0, 2)) <= TOL[dt], n
    if got.get("dS0") is not None:
        assert slice_rel_err(got["dS0"], ref["dS0"], (0, 1)) <= S_TOL


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("T", [1, 2, 16, 17, 31, 32, 33, 63, 64, 65, 96, 97, 128, 200])
def test_lengths(cuda_device, T, N, dt):
    d = make((2, T), 2, 1, N, dt, seed=T + N)
    S0 = state(2, 2, N, T)
    dy, dS = extra((2, T), 2, 2, N, dt, T)
    got = wkv7.delta_backward(*to(d, cuda_device).values(), dy.to(cuda_device), S0.to(cuda_device), dS.to(cuda_device), qk_norm=True)
    check(got, delta.delta_backward(*d.values(), S0, dy, dS, qk_norm=True), dt)
    assert all(got[n].dtype == d["v"].dtype for n in NAMES) and got["dS0"].dtype == torch.float32


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hk,N", [(1, 1, 64), (5, 5, 64), (6, 2, 64), (8, 1, 128), (6, 3, 128)])
@pytest.mark.parametrize("norm", [True, False])
def test_heads(cuda_device, H, Hk, N, dt, norm):
    d = make((1, 150), H, Hk, N, dt, seed=H * 10 + Hk, norm=norm)
    dy, _ = extra((1, 150), 1, H, N, dt, 5)
    got = wkv7.delta_backward(*to(d, cuda_device).values(), dy.to(cuda_device), qk_norm=norm, scale=-0.3)
    check(got, delta.delta_backward(*d.values(), None, dy, None, qk_norm=norm, scale=-0.3), dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N", [64, 128])
def test_packed_sequences(cuda_device, N, dt):
    lens, H, Hk, tail = [37, 0, 1, 64, 130, 0, 5, 96], 4, 2, 11
    cu = [0, *np.cumsum(lens).tolist()]
    d = make((cu[-1] + tail,), H, Hk, N, dt, seed=7)
    dy, dS = extra((cu[-1] + tail,), len(lens), H, N, dt, 8)
    for x in (d["v"], d["k"], dy):
        x[cu[-1]:] = float("nan")
    S0 = state(len(lens), H, N, 3)
    grads = {n: torch.full_like(x, 5.0).to(cuda_device) for n, x in zip(NAMES, (d["q"], d["k"], d["v"], d["g"], d["beta"]))}
    got = wkv7.delta_backward(*to(d, cuda_device).values(), dy.to(cuda_device), S0.to(cuda_device), dS.to(cuda_device),
                              qk_norm=True, grads=grads, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=cuda_device))
    for s, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        ref = delta.delta_backward(*(d[n][a:b][None] for n in TOK), S0[s:s + 1], dy[a:b][None], dS[s:s + 1], qk_norm=True)
        check({**{n: got[n][a:b][None] for n in NAMES}, "dS0": got["dS0"][s:s + 1]}, ref, dt)
    assert all(bool(torch.all(got[n][cu[-1]:] == 5.0)) for n in NAMES)


@pytest.mark.parametrize("cu", [[0, 9, 4, 300], [0, -5, 1000, 300], [100, 5, 70, -3], [300, 0, 300, 300]])
def test_packed_bounds_out_of_order_stay_inside(cuda_device, cu):
    """As forward: every row read or written lies inside the buffers, whose surroundings stay as they were."""
    d = to(make((300,), 2, 1, 64, "bf16", seed=9), cuda_device)
    dy, _ = extra((300,), 3, 2, 64, "bf16", 9)
    pad = {n: torch.full((364, *d[s].shape[1:]), 3.0, dtype=torch.bfloat16, device=cuda_device)
           for n, s in zip(NAMES, TOK)}
    wkv7.delta_backward(*d.values(), dy.to(cuda_device), qk_norm=True, grads={n: x[32:332] for n, x in pad.items()},
                        cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=cuda_device))
    torch.cuda.synchronize()
    for x in pad.values():
        assert bool(torch.all(x[:32] == 3.0)) and bool(torch.all(x[332:] == 3.0))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gates_at_their_ends(cuda_device, dt):
    d = make((2, 100), 3, 3, 64, dt, seed=11, gate=4.0)
    for t, g in ((0, -50.0), (10, float("-inf")), (11, 0.0), (31, float("-inf")), (32, float("-inf")), (63, -300.0),
                 (64, -90.0), (99, 0.0)):
        d["g"][:, t] = g
    d["beta"][:, 20:30] = 0.0
    d["beta"][:, 40:50] = 1.0
    S0 = state(2, 3, 64, 1)
    dy, dS = extra((2, 100), 2, 3, 64, dt, 2)
    got = wkv7.delta_backward(*to(d, cuda_device).values(), dy.to(cuda_device), S0.to(cuda_device), dS.to(cuda_device), qk_norm=True)
    check(got, delta.delta_backward(*d.values(), S0, dy, dS, qk_norm=True), dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_zero_keys_and_queries(cuda_device, dt):
    d = make((1, 70), 2, 2, 64, dt, seed=14)
    d["k"][:, 5:9] = 0.0
    d["q"][:, 8] = 0.0
    dy, _ = extra((1, 70), 1, 2, 64, dt, 3)
    got = wkv7.delta_backward(*to(d, cuda_device).values(), dy.to(cuda_device), qk_norm=True, norm_eps=1e-2)
    check(got, delta.delta_backward(*d.values(), None, dy, None, qk_norm=True, norm_eps=1e-2), dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_strided_rows(cuda_device, dt):
    H, Hk, N, B, T = 4, 2, 64, 2, 75
    d = make((B, T), H, Hk, N, dt, seed=16)
    dy = extra((B, T), B, H, N, dt, 4)[0].to(cuda_device)
    wide = torch.cat([d["q"].flatten(2), d["k"].flatten(2), d["v"].flatten(2)], dim=-1).to(cuda_device)
    q, k, v = wide.split([Hk * N, Hk * N, H * N], dim=-1)
    got = wkv7.delta_backward(q.unflatten(-1, (Hk, N)), k.unflatten(-1, (Hk, N)), v.unflatten(-1, (H, N)),
                              d["g"].to(cuda_device), d["beta"].to(cuda_device), dy, qk_norm=True)
    ref = wkv7.delta_backward(*to(d, cuda_device).values(), dy, qk_norm=True)
    for n in NAMES + ("dS0",):
        assert torch.equal(got[n], ref[n]), n


def test_against_differences(cuda_device):
    """fp32: the directional derivative of <dy, y> + <dS_T, S_T> along random directions, by central
    differences of the GPU forward. The forward's values carry about 1e-6 of rounding over a
    loss of order 1, which a step of 2e-2 turns into 1e-4 of the slope; the third-order term of the
    difference is of order h^2 = 4e-4 of it."""
    B, T, H, Hk, N = 1, 70, 2, 1, 64
    d = make((B, T), H, Hk, N, "f32", seed=41)
    S0 = state(B, H, N, 2)
    dy, dS = extra((B, T), B, H, N, "f32", 6)
    x = {**to(d, cuda_device), "S0": S0.to(cuda_device)}
    dy, dS = dy.to(cuda_device) / 100, dS.to(cuda_device) / 10
    got = wkv7.delta_backward(*(x[n] for n in TOK), dy, x["S0"], dS, qk_norm=True)

    def loss(y):
        out, S = wkv7.delta_forward(*(y[n] for n in TOK), y["S0"], qk_norm=True)
        return float((out.double() * dy).sum() + (S.double() * dS).sum())

    g = torch.Generator().manual_seed(3)
    for n, s in (("q", 1.0), ("k", 1.0), ("v", 1.0), ("g", 0.3), ("beta", 0.3), ("S0", 0.3)):
        way = (s * torch.randn(x[n].shape, generator=g)).to(cuda_device)
        h = 2e-2
        slope = (loss({**x, n: x[n] + h * way}) - loss({**x, n: x[n] - h * way})) / (2 * h)
        want = float((got["d" + n].double() * way).sum())
        size = float((got["d" + n].double().norm() * way.double().norm()))
        assert abs(slope - want) <= 2e-3 * size, (n, slope, want, size)


def test_state_gradient_in_place_and_optional(cuda_device):
    d = to(make((2, 60), 2, 2, 64, "bf16", seed=19), cuda_device)
    dy, dS = (x.to(cuda_device) for x in extra((2, 60), 2, 2, 64, "bf16", 7))
    ref = wkv7.delta_backward(*d.values(), dy, None, dS, qk_norm=True)
    none = wkv7.delta_backward(*d.values(), dy, None, dS, qk_norm=True, return_state_grad=False)
    assert none["dS0"] is None and all(torch.equal(none[n], ref[n]) for n in NAMES)
    buf = dS.clone()
    got = wkv7.delta_backward(*d.values(), dy, None, buf, qk_norm=True, dS0=buf)
    assert got["dS0"] is buf and torch.equal(buf, ref["dS0"]) and all(torch.equal(got[n], ref[n]) for n in NAMES)


def test_without_tokens(cuda_device):
    d = to(make((2, 0), 2, 2, 64, "bf16", seed=18), cuda_device)
    dS = state(2, 2, 64, 5).to(cuda_device)
    got = wkv7.delta_backward(*d.values(), torch.empty_like(d["v"]), None, dS)
    assert got["dq"].shape == (2, 0, 2, 64) and torch.equal(got["dS0"], dS)
    assert bool(torch.all(wkv7.delta_backward(*d.values(), torch.empty_like(d["v"]))["dS0"] == 0))


def test_repeats_other_streams_and_graphs(cuda_device):
    """Bit for bit: again, on a stream of the caller's, from a captured graph on new inputs, and with a
    workspace full of NaN."""
    d, d2 = (to(make((2, 130), 4, 2, 64, "bf16", seed=s), cuda_device) for s in (20, 21))
    dy, dS = (x.to(cuda_device) for x in extra((2, 130), 2, 4, 64, "bf16", 7))
    ref, ref2 = (wkv7.delta_backward(*x.values(), dy, None, dS, qk_norm=True) for x in (d, d2))
    need = wkv7.load().wkv7_delta_backward_workspace_bytes(2, 130, 4, 2, 64, wkv7.BF16, None)
    ws = torch.full((need // 4,), float("nan"), device=cuda_device)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for got in (wkv7.delta_backward(*d.values(), dy, None, dS, qk_norm=True),
                wkv7.delta_backward(*d.values(), dy, None, dS, qk_norm=True, workspace=ws),
                wkv7.delta_backward(*d.values(), dy, None, dS, qk_norm=True, stream=s)):
        torch.cuda.synchronize()
        for n in NAMES + ("dS0",):
            assert torch.equal(got[n], ref[n]), n
    held = {n: x.clone() for n, x in d.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = wkv7.delta_backward(*held.values(), dy, None, dS, qk_norm=True)
    for n in TOK:
        held[n].copy_(d2[n])
    graph.replay()
    torch.cuda.synchronize()
    for n in NAMES + ("dS0",):
        assert torch.equal(got[n], ref2[n]), n


@pytest.mark.parametrize("N,H,Hk", [(64, 8, 4), (64, 3, 3), (128, 4, 2)])
def test_more_chunks_than_the_gpu_holds_at_once(cuda_device, N, H, Hk):
    """A CTA of the gradients' kernel takes several chunks, over the ends of sequences, empty ones among them."""
    lens = [900, 0, 1, 1500, 63, 0, 64, 1400, 65, 0]
    cu = [0, *np.cumsum(lens).tolist()]
    d = make((cu[-1],), H, Hk, N, "bf16", seed=61)
    dy, dS = extra((cu[-1],), len(lens), H, N, "bf16", 62)
    S0 = state(len(lens), H, N, 63)
    got = wkv7.delta_backward(*to(d, cuda_device).values(), dy.to(cuda_device), S0.to(cuda_device), dS.to(cuda_device),
                              qk_norm=True, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=cuda_device))
    for s, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        ref = delta.delta_backward(*(d[n][a:b][None] for n in TOK), S0[s:s + 1], dy[a:b][None], dS[s:s + 1], qk_norm=True)
        check({**{n: got[n][a:b][None] for n in NAMES}, "dS0": got["dS0"][s:s + 1]}, ref, "bf16")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_nan_stays_in_its_sequence_and_key_head(cuda_device, dt):
    """A NaN value reaches no gradient of another sequence, nor dv, dg or dbeta of another head."""
    d = make((3, 150), 4, 2, 64, dt, seed=64)
    dy, dS = extra((3, 150), 3, 4, 64, dt, 65)
    run = lambda: wkv7.delta_backward(*to(d, cuda_device).values(), dy.to(cuda_device), None, dS.to(cuda_device),  # noqa: E731
                                      qk_norm=True)
    clean = run()
    d["v"][1, 70, 1, 5] = float("nan")
    got = run()
    for n in NAMES + ("dS0",):
        assert torch.equal(got[n][[0, 2]], clean[n][[0, 2]]), n
    for n in ("dv", "dg", "dbeta", "dS0"):
        x, y = (t[n][1] if n == "dS0" else t[n][1].transpose(0, 1) for t in (got, clean))
        assert torch.equal(x[[0, 2, 3]], y[[0, 2, 3]]), n
    for n in ("dq", "dk"):
        assert torch.equal(got[n][1, :, 1], clean[n][1, :, 1]), n
    assert not torch.isfinite(got["dbeta"][1, 70, 1])


def test_two_calls_at_once(cuda_device):
    """On two streams, each with its own workspace: the same bits as one after the other."""
    a, b = (to(make((4, 500), 6, 3, 64, "bf16", seed=s), cuda_device) for s in (66, 67))
    dy = extra((4, 500), 4, 6, 64, "bf16", 68)[0].to(cuda_device)
    ref = [wkv7.delta_backward(*x.values(), dy, qk_norm=True) for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [wkv7.delta_backward(*x.values(), dy, qk_norm=True, stream=s) for x, s in zip((a, b), streams)]
    torch.cuda.synchronize()
    for g, r in zip(got, ref):
        for n in NAMES + ("dS0",):
            assert torch.equal(g[n], r[n]), n


def test_training_step_follows_the_oracle(cuda_device):
    """Forward and backward as a step uses them: a loss on y and the state, split over two calls with
    the state and its gradient handed between them, equals the oracle's gradients of one pass."""
    B, T, H, Hk, N, cut = 2, 140, 4, 2, 64, 77
    d = make((B, T), H, Hk, N, "bf16", seed=51)
    dy, dS = extra((B, T), B, H, N, "bf16", 9)
    x = to(d, cuda_device)
    first, second = ({n: t[:, a:b].contiguous() for n, t in x.items()} for a, b in ((0, cut), (cut, T)))
    _, S = wkv7.delta_forward(*first.values(), qk_norm=True)
    dyd = dy.to(cuda_device)
    g2 = wkv7.delta_backward(*second.values(), dyd[:, cut:].contiguous(), S, dS.to(cuda_device), qk_norm=True)
    g1 = wkv7.delta_backward(*first.values(), dyd[:, :cut].contiguous(), None, g2["dS0"], qk_norm=True)
    got = {n: torch.cat([g1[n], g2[n]], 1) for n in NAMES}
    ref = delta.delta_backward(*d.values(), None, dy, dS, qk_norm=True)
    check({**got, "dS0": g1["dS0"]}, ref, "bf16")
