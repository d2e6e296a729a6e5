"""The gated delta rule on the GPU against the fp64 oracle: forward and single-token step."""
import numpy as np
import pytest
import torch

from linear_rnn_sequence_rwkv_b200 import wkv7
from oracle import delta
from tests.delta_util import S_TOL, TOK, Y_TOL, make, s_err, state, y_err

pytestmark = pytest.mark.gpu


def to(d, dev):
    return {n: x.to(dev) for n, x in d.items()}


def check(y, S, yr, Sr, dt):
    assert S is None or s_err(S, Sr) <= S_TOL
    if yr.size:
        assert y_err(y, yr) <= Y_TOL[dt]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 200])
def test_forward_lengths(cuda_device, T, N, dt):
    d = make((2, T), 2, 1, N, dt, seed=T + N)
    S0 = state(2, 2, N, T)
    y, S = wkv7.delta_forward(*to(d, cuda_device).values(), S0.to(cuda_device), qk_norm=True)
    yr, Sr = delta.delta_recurrence(*d.values(), S0, qk_norm=True)
    assert y.dtype == d["v"].dtype and S.dtype == torch.float32
    check(y, S, yr, Sr, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hk,N", [(1, 1, 64), (5, 5, 64), (6, 2, 64), (8, 1, 128), (6, 3, 128)])
@pytest.mark.parametrize("norm", [True, False])
def test_forward_heads(cuda_device, H, Hk, N, dt, norm):
    d = make((1, 77), H, Hk, N, dt, seed=H * 10 + Hk, norm=norm)
    y, S = wkv7.delta_forward(*to(d, cuda_device).values(), qk_norm=norm, scale=0.3)
    check(y, S, *delta.delta_recurrence(*d.values(), qk_norm=norm, scale=0.3), dt)


def _cu(lens):
    return [0, *np.cumsum(lens).tolist()]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N", [64, 128])
def test_forward_packed_sequences(cuda_device, N, dt):
    """Ragged lengths with empty sequences among them; rows behind the last one stay as they were."""
    lens, H, Hk, tail = [37, 0, 1, 64, 130, 0, 5, 96], 4, 2, 11
    cu = _cu(lens)
    d = make((cu[-1] + tail,), H, Hk, N, dt, seed=7)
    d["v"][cu[-1]:] = float("nan")
    d["k"][cu[-1]:] = float("inf")
    S0 = state(len(lens), H, N, 3)
    y = torch.full_like(d["v"], 5.0).to(cuda_device)
    _, S = wkv7.delta_forward(*to(d, cuda_device).values(), S0.to(cuda_device), qk_norm=True, y=y,
                              cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=cuda_device))
    for s, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        yr, Sr = delta.delta_recurrence(*(d[n][a:b][None] for n in TOK), S0[s:s + 1], qk_norm=True)
        check(y[a:b][None], S[s:s + 1], yr, Sr, dt)
    assert torch.all(y[cu[-1]:] == 5.0)


def test_packed_without_an_output_has_zero_rows_behind(cuda_device):
    d = make((20,), 2, 2, 64, "bf16", seed=8)
    cu = torch.tensor([0, 12], dtype=torch.int32, device=cuda_device)
    y, S = wkv7.delta_forward(*to(d, cuda_device).values(), cu_seqlens=cu, qk_norm=True)
    assert torch.all(y[12:] == 0) and S.shape == (1, 2, 64, 64)


@pytest.mark.parametrize("cu", [[0, 9, 4, 30], [0, -5, 1000, 30], [10, 5, 7, -3]])
def test_packed_bounds_out_of_order_stay_inside(cuda_device, cu):
    """Entries outside 0..T or decreasing are clamped: every row that is read or written lies inside."""
    d = make((30,), 2, 1, 64, "bf16", seed=9)
    y, S = wkv7.delta_forward(*to(d, cuda_device).values(), qk_norm=True,
                              cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=cuda_device))
    torch.cuda.synchronize()
    assert y.shape == d["v"].shape and bool(torch.isfinite(S).all())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_forward_gates_at_their_ends(cuda_device, dt):
    """Log decays of 0, very negative ones and -inf (the state is reset), strengths of 0 and 1."""
    d = make((2, 100), 3, 3, 64, dt, seed=11, gate=4.0)
    for t, g in ((0, -50.0), (10, float("-inf")), (11, 0.0), (31, float("-inf")), (32, float("-inf")), (63, -300.0),
                 (64, -90.0), (99, 0.0)):
        d["g"][:, t] = g
    d["beta"][:, 20:30] = 0.0
    d["beta"][:, 40:50] = 1.0
    S0 = state(2, 3, 64, 1)
    y, S = wkv7.delta_forward(*to(d, cuda_device).values(), S0.to(cuda_device), qk_norm=True)
    check(y, S, *delta.delta_recurrence(*d.values(), S0, qk_norm=True), dt)


def test_forward_steep_gates_keep_their_neighbours(cuda_device):
    """Sums of log decays reach the thousands inside a chunk; the decays between neighbours, which
    are differences of such sums, must keep fp32 accuracy."""
    d = make((1, 192), 2, 2, 64, "f32", seed=12)
    d["g"][:, ::2] = -100.25
    d["g"][:, 1::2] = -0.001953125
    y, S = wkv7.delta_forward(*to(d, cuda_device).values(), qk_norm=True)
    check(y, S, *delta.delta_recurrence(*d.values(), qk_norm=True), "f32")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_forward_repeated_keys(cuda_device, dt):
    """One key throughout, written with full strength: the system inside a chunk is as far from
    the identity as it gets (every product of keys is 1)."""
    d = make((1, 96), 2, 2, 64, dt, seed=13, gate=0.01)
    d["k"][:] = d["k"][:, :1]
    d["beta"][:] = 1.0
    y, S = wkv7.delta_forward(*to(d, cuda_device).values(), qk_norm=True)
    check(y, S, *delta.delta_recurrence(*d.values(), qk_norm=True), dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_forward_zero_keys_and_large_values(cuda_device, dt):
    d = make((1, 70), 2, 2, 64, dt, seed=14)
    d["k"][:, 5:9] = 0.0
    d["q"][:, 8] = 0.0
    d["v"] *= 2.0 ** 40
    y, S = wkv7.delta_forward(*to(d, cuda_device).values(), qk_norm=True)
    check(y, S, *delta.delta_recurrence(*d.values(), qk_norm=True), dt)


def test_forward_nan_stays_in_its_sequence_and_head(cuda_device):
    d = make((2, 70), 2, 2, 64, "bf16", seed=15)
    d["v"][1, 40, 1, 3] = float("nan")
    y, S = wkv7.delta_forward(*to(d, cuda_device).values(), qk_norm=True)
    yr, Sr = delta.delta_recurrence(*(x[:1] for x in d.values()), qk_norm=True)
    check(y[:1], S[:1], yr, Sr, "bf16")
    assert torch.isfinite(y[1, :, 0]).all() and torch.isfinite(y[1, :40, 1]).all()
    assert torch.isnan(y[1, 40:, 1, 3]).all() and torch.isfinite(y[1, :, 1, :3]).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("t", [0, 45, 99])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_forward_inputs_that_are_not_finite(cuda_device, bad, t, N, dt):
    """Each reaches its own token and later ones of what it belongs to, and nothing else."""
    d = make((2, 100), 4, 2, N, dt, seed=17)
    ref, S_ref = wkv7.delta_forward(*to(d, cuda_device).values(), qk_norm=True)
    for name, heads in (("q", [2, 3]), ("k", [2, 3]), ("v", [2]), ("g", [2]), ("beta", [2])):
        x = {n: v.clone() for n, v in d.items()}
        if name in "qk":
            x[name][1, t, 1, 7] = bad
        elif name == "v":
            x[name][1, t, 2, 7] = bad
        else:
            x[name][1, t, 2] = bad
        y, S = wkv7.delta_forward(*to(x, cuda_device).values(), qk_norm=True)
        other = [h for h in range(4) if h not in heads]
        assert torch.equal(y[0], ref[0]) and torch.equal(S[0], S_ref[0]), name
        assert torch.equal(y[1][:, other], ref[1][:, other]) and torch.equal(S[1, other], S_ref[1, other]), name
        mine, was = y[1][:, heads], ref[1][:, heads]
        for part in ((mine[:t], was[:t]), *([(mine[t + 1:], was[t + 1:])] if name == "q" else [])):
            assert float((part[0] - part[1]).abs().max() if part[0].numel() else 0) <= Y_TOL[dt] * float(was.abs().max()), name
        if name == "q":
            assert not torch.isfinite(mine[t]).any()
            assert torch.equal(S[1], S_ref[1])
        elif name == "v":
            assert not torch.isfinite(mine[t:, :, 7]).any() and not torch.isfinite(S[1, 2, 7]).any()
            mine, was = (z[..., [i for i in range(N) if i != 7]] for z in (mine, was))
            assert float((mine - was).abs().max()) <= Y_TOL[dt] * float(was.abs().max())
        else:
            assert not torch.isfinite(mine[t:]).any() and not torch.isfinite(S[1, heads]).any()


def test_forward_two_calls_at_once(cuda_device):
    a, b = (to(make((4, 500), 6, 3, 64, "bf16", seed=s), cuda_device) for s in (18, 19))
    ref = [wkv7.delta_forward(*x.values(), qk_norm=True) for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [wkv7.delta_forward(*x.values(), qk_norm=True, stream=s) for x, s in zip((a, b), streams)]
    torch.cuda.synchronize()
    for g, r in zip(got, ref):
        assert torch.equal(g[0], r[0]) and torch.equal(g[1], r[1])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_forward_strided_rows(cuda_device, dt):
    """q, k and v as views of one projection's output, rows wider than their own heads."""
    H, Hk, N, B, T = 4, 2, 64, 2, 75
    d = make((B, T), H, Hk, N, dt, seed=16)
    wide = torch.cat([d["q"].flatten(2), d["k"].flatten(2), d["v"].flatten(2)], dim=-1).to(cuda_device)
    q, k, v = wide.split([Hk * N, Hk * N, H * N], dim=-1)
    q, k, v = q.unflatten(-1, (Hk, N)), k.unflatten(-1, (Hk, N)), v.unflatten(-1, (H, N))
    assert not v.is_contiguous()
    g, b = d["g"].to(cuda_device), d["beta"].to(cuda_device)
    y, S = wkv7.delta_forward(q, k, v, g, b, qk_norm=True)
    y2, S2 = wkv7.delta_forward(*to(d, cuda_device).values(), qk_norm=True)
    assert torch.equal(y, y2) and torch.equal(S, S2)
    pool = torch.zeros(B, H, N, N, device=cuda_device)
    y3 = wkv7.delta_step(q[:, 0], k[:, 0], v[:, 0], g[:, 0].contiguous(), b[:, 0].contiguous(), pool, qk_norm=True)
    check(y3[:, None], None, delta.delta_recurrence(*(x[:, :1] for x in d.values()), qk_norm=True)[0], None, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_split_with_state_hand_off_equals_one_pass(cuda_device, dt):
    """Cut where no chunk ends, the state handed on in place."""
    d = to(make((2, 150), 2, 2, 64, dt, seed=17), cuda_device)
    y, S = wkv7.delta_forward(*d.values(), qk_norm=True)
    S1 = torch.zeros_like(S)
    parts = []
    for a, b in ((0, 41), (41, 42), (42, 150)):
        yp, _ = wkv7.delta_forward(*(x[:, a:b].contiguous() for x in d.values()), S1, S_T=S1, qk_norm=True)
        parts.append(yp)
    check(torch.cat(parts, 1), S1, y.double().cpu().numpy(), S.double().cpu().numpy(), dt)


def test_forward_without_tokens_hands_the_state_on(cuda_device):
    d = to(make((2, 0), 2, 2, 64, "bf16", seed=18), cuda_device)
    S0 = state(2, 2, 64, 5).to(cuda_device)
    y, S = wkv7.delta_forward(*d.values(), S0)
    assert y.shape == (2, 0, 2, 64) and torch.equal(S, S0)
    _, S = wkv7.delta_forward(*d.values())
    assert torch.all(S == 0)


def test_forward_optional_outputs(cuda_device):
    d = to(make((1, 40), 2, 2, 64, "bf16", seed=19), cuda_device)
    y, S = wkv7.delta_forward(*d.values(), qk_norm=True)
    y2, S2 = wkv7.delta_forward(*d.values(), qk_norm=True, return_state=False)
    assert S2 is None and torch.equal(y, y2)


def test_forward_on_another_stream_and_in_a_graph(cuda_device):
    """The same bits on a stream of the caller's, and from a captured graph replayed on new inputs."""
    d = to(make((2, 90), 2, 1, 64, "bf16", seed=20), cuda_device)
    d2 = to(make((2, 90), 2, 1, 64, "bf16", seed=21), cuda_device)
    ref, ref2 = (wkv7.delta_forward(*x.values(), qk_norm=True) for x in (d, d2))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, S = wkv7.delta_forward(*d.values(), qk_norm=True, stream=s)
    s.synchronize()
    assert torch.equal(y, ref[0]) and torch.equal(S, ref[1])
    held = {n: x.clone() for n, x in d.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, S = wkv7.delta_forward(*held.values(), qk_norm=True)
    for n in TOK:
        held[n].copy_(d2[n])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, ref2[0]) and torch.equal(S, ref2[1])


def test_forward_repeats_bit_for_bit(cuda_device):
    d = to(make((3, 333), 4, 2, 128, "bf16", seed=22), cuda_device)
    y, S = wkv7.delta_forward(*d.values(), qk_norm=True)
    for _ in range(3):
        y2, S2 = wkv7.delta_forward(*d.values(), qk_norm=True)
        assert torch.equal(y, y2) and torch.equal(S, S2)


def test_forward_rows_past_32_bit_offsets(cuda_device):
    """2^31 elements of v lie before the second sequence."""
    H, N, T = 64, 128, 262_144 + 40
    if torch.cuda.mem_get_info()[0] < 40e9:
        pytest.skip("needs 40 GB")
    d = make((2, 40), H, 1, N, "bf16", seed=23)
    rows = 2 * T
    q = torch.zeros(rows, 1, N, device=cuda_device, dtype=torch.bfloat16)
    v = torch.zeros(rows, H, N, device=cuda_device, dtype=torch.bfloat16)
    g = torch.full((rows, H), -1.0, device=cuda_device, dtype=torch.bfloat16)
    k, b = torch.zeros_like(q), torch.zeros_like(g)
    for n, x in zip(TOK, (q, k, v, g, b)):
        x[rows - 40:] = d[n][1].to(cuda_device)
    cu = torch.tensor([0, rows - 40, rows], dtype=torch.int32, device=cuda_device)
    y, S = wkv7.delta_forward(q, k, v, g, b, cu_seqlens=cu, qk_norm=True)
    check(y[rows - 40:][None], S[1:], *delta.delta_recurrence(*(d[n][1:] for n in TOK), qk_norm=True), "bf16")


# ---- one token ---------------------------------------------------------------------------------

@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,Hk,N", [(1, 1, 1, 64), (3, 4, 2, 64), (7, 3, 1, 128), (2, 5, 5, 128)])
@pytest.mark.parametrize("norm", [True, False])
def test_step(cuda_device, B, H, Hk, N, dt, norm):
    d = make((B,), H, Hk, N, dt, seed=B + N, norm=norm)
    S0 = state(B, H, N, 9)
    S = S0.to(cuda_device)
    y = wkv7.delta_step(*to(d, cuda_device).values(), S, qk_norm=norm)
    yr, Sr = delta.delta_recurrence(*(x[:, None] for x in d.values()), S0, qk_norm=norm)
    check(y[:, None], S, yr, Sr, dt)


@pytest.mark.parametrize("N", [64, 128])
def test_step_on_a_pool(cuda_device, N):
    """Slots in any order, padding, values outside the pool; states that no row names stay as they were."""
    B, H, pool = 9, 2, 20
    d = make((B,), H, H, N, "bf16", seed=31)
    slots = [4, -1, 19, 0, 20, 7, -2147483648, 11, 2147483647]
    S0 = state(pool, H, N, 10)
    S = S0.to(cuda_device)
    y = wkv7.delta_step(*to(d, cuda_device).values(), S, qk_norm=True,
                        slots=torch.tensor(slots, dtype=torch.int32, device=cuda_device))
    live = [b for b, s in enumerate(slots) if 0 <= s < pool]
    at = [slots[b] for b in live]
    yr, Sr = delta.delta_recurrence(*(x[live][:, None] for x in d.values()), S0[at], qk_norm=True)
    check(y[live][:, None], S[at], yr, Sr, "bf16")
    rest = [s for s in range(pool) if s not in at]
    assert torch.equal(S[rest].cpu(), S0[rest])
    assert torch.all(y[[b for b in range(B) if b not in live]] == 0)


def test_step_rows_that_share_a_slot_follow_one_another(cuda_device):
    B, H, N = 300, 2, 64
    d = make((B,), H, H, N, "f32", seed=32)
    g = torch.Generator().manual_seed(1)
    slots = torch.randint(0, 40, (B,), generator=g, dtype=torch.int32)
    S0 = state(40, H, N, 11)
    S = S0.to(cuda_device)
    y = wkv7.delta_step(*to(d, cuda_device).values(), S, qk_norm=True, slots=slots.to(cuda_device))
    for s in range(40):
        rows = (slots == s).nonzero().flatten().tolist()
        if not rows:
            assert torch.equal(S[s].cpu(), S0[s])
            continue
        yr, Sr = delta.delta_recurrence(*(d[n][rows][None] for n in TOK), S0[s:s + 1], qk_norm=True)
        check(y[rows][None], S[s:s + 1], yr, Sr, "f32")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_step_rows_that_share_a_slot_at_head_size_128(cuda_device, dt):
    B, H, N = 37, 2, 128
    d = make((B,), H, 1, N, dt, seed=35)
    slots = torch.tensor([(3 * b) % 7 - 1 for b in range(B)], dtype=torch.int32)
    S0 = state(6, H, N, 13)
    S = S0.to(cuda_device)
    y = wkv7.delta_step(*to(d, cuda_device).values(), S, qk_norm=True, slots=slots.to(cuda_device))
    assert bool(torch.all(y[slots.to(cuda_device) < 0] == 0))
    for s in range(6):
        rows = (slots == s).nonzero().flatten().tolist()
        yr, Sr = delta.delta_recurrence(*(d[n][rows][None] for n in TOK), S0[s:s + 1], qk_norm=True)
        check(y[rows][None], S[s:s + 1], yr, Sr, dt)


def test_steps_equal_the_forward(cuda_device):
    """Prefill, then 20 steps from a captured graph, against one forward over all tokens."""
    B, T, H, N = 3, 60, 4, 64
    d = to(make((B, T), H, 2, N, "bf16", seed=33), cuda_device)
    y, S = wkv7.delta_forward(*d.values(), qk_norm=True)
    yp, Sp = wkv7.delta_forward(*(x[:, :40].contiguous() for x in d.values()), qk_norm=True)
    one = {n: x[:, 40].contiguous() for n, x in d.items()}
    keep = Sp.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ys = wkv7.delta_step(*one.values(), Sp, qk_norm=True)
    Sp.copy_(keep)
    outs = [yp]
    for t in range(40, T):
        for n in TOK:
            one[n].copy_(d[n][:, t])
        graph.replay()
        outs.append(ys[:, None].clone())
    check(torch.cat(outs, 1), Sp, y.double().cpu().numpy(), S.double().cpu().numpy(), "bf16")


def test_step_on_a_pool_past_32_bit_offsets(cuda_device):
    N, H, pool = 128, 1, 131_072 + 8        # 2^31 elements lie before the last eight states
    if torch.cuda.mem_get_info()[0] < 20e9:
        pytest.skip("needs 20 GB")
    d = make((2,), H, H, N, "bf16", seed=34)
    S = torch.zeros(pool, H, N, N, device=cuda_device)
    S0 = state(2, H, N, 12)
    at = [pool - 1, pool - 3]
    S[at] = S0.to(cuda_device)
    y = wkv7.delta_step(*to(d, cuda_device).values(), S, qk_norm=True,
                        slots=torch.tensor(at, dtype=torch.int32, device=cuda_device))
    yr, Sr = delta.delta_recurrence(*(x[:, None] for x in d.values()), S0, qk_norm=True)
    check(y[:, None], S[at], yr, Sr, "bf16")
