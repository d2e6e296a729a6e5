"""Beam selection and the reordering of states on the GPU against the oracle, and a decoding loop."""
import numpy as np
import pytest
import torch

from linear_rnn_sequence_rwkv_b200 import wkv7
from oracle import delta
from tests.delta_util import DT, Y_TOL, make, s_err, y_err

pytestmark = pytest.mark.gpu
S_TOL = 2e-6   # scores: fp32's rounding of a value up to 50 (2^-24 * 50 = 3e-6 at most, in absolute
               # terms; compared relative to the largest score, 2^-24 plus the normaliser's own 1e-7)


def pick(dev, x, s, M, finished=None, eos=0, **kw):
    out = wkv7.beam_select(x.to(dev), s.to(dev), M, eos=eos, **kw,
                           finished=None if finished is None else finished.to(dev))
    return [t.cpu().numpy() for t in out]


def check(dev, x, s, M, finished=None, eos=0):
    got = pick(dev, x, s, M, finished, eos)
    ref = delta.beam_select(x.double().numpy(), s.numpy(), M, None if finished is None else finished.numpy(), eos)
    np.testing.assert_array_equal(got[1], ref[1])
    np.testing.assert_array_equal(got[2], ref[2])
    fin = np.isfinite(ref[0])
    assert np.array_equal(got[0][~fin], ref[0][~fin])
    if fin.any():
        assert np.max(np.abs(got[0][fin] - ref[0][fin])) <= S_TOL * max(1.0, np.max(np.abs(ref[0][fin])))


def draw(B, K, V, dt, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn(B, K, V, generator=g)).to(DT[dt]), -20 + 2 * torch.randn(B, K, generator=g)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,K,V,M", [(1, 1, 1, 1), (1, 1, 1, 3), (2, 3, 5, 15), (2, 3, 5, 16), (3, 4, 255, 8), (1, 2, 2047, 64),
                                     (2, 64, 33, 64), (1, 4, 8192, 8), (2, 3, 8193, 5), (1, 5, 50277, 10), (40, 8, 9001, 16),
                                     (1, 1, 200003, 64)])
def test_select(cuda_device, B, K, V, M, dt):
    check(cuda_device, *draw(B, K, V, dt, B + V), M)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,K,V,M", [(1, 64, 50277, 64), (1, 2, 600_011, 33), (3, 33, 20_000, 7)])
def test_select_many_lists(cuda_device, B, K, V, M, dt):
    """More lists than fit shared memory, more than a warp has lanes for, more rows than lanes."""
    check(cuda_device, *draw(B, K, V, dt, B + V), M)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_select_ties_between_rows_go_to_the_lowest_beam(cuda_device, dt):
    """64 equal rows with equal scores: every place is a tie between all beams."""
    x, _ = draw(1, 1, 3001, dt, 9)
    check(cuda_device, x.expand(1, 64, 3001).contiguous(), torch.zeros(1, 64), 64)
    check(cuda_device, x.expand(1, 40, 3001).contiguous(), (torch.arange(40) % 3 - 1).float()[None], 50)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_select_ties_go_to_the_lowest_index(cuda_device, dt):
    """Equal logits everywhere, and a few distinct values in coarse steps."""
    x, s = draw(2, 3, 20011, dt, 5)
    check(cuda_device, torch.zeros_like(x), torch.zeros_like(s), 17)
    check(cuda_device, torch.round(x / 4), torch.full_like(s, -1.0), 64)
    y = torch.full_like(x, -5.0)
    y[:, :, 9000:9100] = -0.0
    y[:, :, 9050:9060] = 0.0                          # -0 and +0 are one score
    check(cuda_device, y, torch.zeros_like(s), 64)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_select_masked_and_bad_rows(cuda_device, dt):
    """Masks of -inf and of the type's lowest value, NaN, rows with nothing, +inf, dead beams."""
    x, s = draw(6, 4, 3001, dt, 6)
    lowest = torch.finfo(DT[dt]).min
    x[0, :, 100:] = float("-inf")
    x[0, 1, :] = float("-inf")
    x[1, :, 50:] = lowest
    x[2, 0, ::3] = float("nan")
    x[2, 1, :] = float("nan")
    x[3, 2, 77] = float("inf")
    x[3, 3, :] = lowest
    s[4] = float("-inf")
    s[4, 2] = -3.0
    s[5, 1] = float("nan")
    s[5, 3] = float("-inf")
    check(cuda_device, x, s, 13)
    x[:] = float("-inf")
    got = pick(cuda_device, x, s, 3)
    assert np.all(np.isneginf(got[0])) and np.all(got[1] == -1) and np.all(got[2] == -1)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [(1, 2), (40, 16)])       # one block per CTA, and a whole row
@pytest.mark.parametrize("M", [1, 16, 33, 64])
def test_select_orders_that_fill_the_buffer(cuda_device, rows, M, dt):
    """Rising logits (every block holds only better ones), rising in steps of equal values, falling, all
    equal, and a few tokens among masked ones: what is gathered overflows, or the floor never rises."""
    B, K = rows
    V = 40_003
    up = torch.arange(V, dtype=torch.float32) / 400
    kinds = [up, torch.floor(up), -up, torch.zeros(V), torch.where(torch.arange(V) % 3001 == 0, up, float("-inf")),
             torch.where(torch.arange(V) < 9000, float("-inf"), torch.floor(up)),
             torch.where(torch.arange(V) > 20000, torch.tensor(torch.finfo(DT[dt]).min), torch.zeros(()))]
    x = torch.stack([kinds[i % len(kinds)] for i in range(B * K)]).reshape(B, K, V).to(DT[dt])
    s = torch.arange(B * K, dtype=torch.float32).reshape(B, K) / 8
    got = pick(cuda_device, x, s, M)
    some = range(B) if B < 8 else (0, 1, 2, 3, B - 1)
    ref = delta.beam_select(x[list(some)].double().numpy(), s[list(some)].numpy(), M)
    np.testing.assert_array_equal(got[1][list(some)], ref[1])
    np.testing.assert_array_equal(got[2][list(some)], ref[2])


def test_select_few_tokens_left(cuda_device):
    """Fewer continuations than picks: the rest say so."""
    x, s = draw(1, 2, 5000, "f32", 7)
    x[0, 0, :] = float("-inf")
    x[0, 1, 3:] = float("-inf")
    check(cuda_device, x, s, 8)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_select_finished_beams(cuda_device, dt):
    x, s = draw(5, 6, 777, dt, 8)
    f = torch.rand(5, 6, generator=torch.Generator().manual_seed(1)) < 0.5
    f[0] = True
    f[1] = False
    x[f] = float("nan")                               # nothing of a finished beam's logits is used
    s[2, 0] = float("-inf")
    check(cuda_device, x, s, 12, f, eos=776)
    u8 = pick(cuda_device, x, s, 12, f.to(torch.uint8), eos=776)
    assert np.array_equal(u8[2], pick(cuda_device, x, s, 12, f, eos=776)[2])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_select_large_logits(cuda_device, dt):
    x, s = draw(2, 3, 4099, dt, 9, spread=300.0)
    check(cuda_device, x, s, 6)


def test_select_strided_rows_and_out(cuda_device):
    """Rows of a padded vocabulary, at every alignment; outputs and workspace of the caller's."""
    x, s = draw(2, 3, 1000, "bf16", 10)
    ref = pick(cuda_device, x, s, 7)
    wide = torch.full((2, 3, 1029), 99.0, dtype=torch.bfloat16)
    wide[..., :1000] = x
    w = wide.to(cuda_device)
    out = (torch.empty(2, 7, device=cuda_device), *(torch.empty(2, 7, dtype=torch.int32, device=cuda_device) for _ in "pt"))
    got = wkv7.beam_select(w[..., :1000], s.to(cuda_device), 7, out=out,
                           workspace=torch.empty(1 << 20, dtype=torch.uint8, device=cuda_device))
    assert all(a is b for a, b in zip(got, out))
    for a, b in zip(got, ref):
        assert np.array_equal(a.cpu().numpy(), b)


def test_select_rows_past_32_bit_offsets(cuda_device):
    B, K, V = 530, 64, 65536                          # 2.2e9 logits
    if torch.cuda.mem_get_info()[0] < 20e9:
        pytest.skip("needs 20 GB")
    x = torch.zeros(B, K, V, dtype=torch.bfloat16, device=cuda_device)
    s = torch.zeros(B, K, device=cuda_device)
    small, _ = draw(1, K, V, "bf16", 11)
    x[-1] = small[0].to(cuda_device)
    got = wkv7.beam_select(x, s, 4)
    ref = delta.beam_select(small.double().numpy(), np.zeros((1, K)), 4)
    assert np.array_equal(got[2][-1].cpu().numpy(), ref[2][0]) and np.array_equal(got[1][-1].cpu().numpy(), ref[1][0])


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("L,B,K,shape,dtype", [(1, 1, 1, (4,), torch.float32), (2, 3, 4, (2, 64, 64), torch.float32),
                                               (1, 5, 7, (24,), torch.bfloat16), (3, 2, 16, (1000,), torch.float32),
                                               (1, 2, 31, (16,), torch.uint8), (2, 2, 64, (1028,), torch.float32)])
def test_reorder(cuda_device, L, B, K, shape, dtype, in_place):
    g = torch.Generator().manual_seed(K)
    x = torch.randint(0, 100, (L, B, K, *shape), generator=g).to(dtype)
    p = torch.randint(0, K, (B, K), generator=g, dtype=torch.int32)
    p[0, 0] = -1                                       # stays
    if B > 1:
        p[1] = torch.randperm(K, generator=g).to(torch.int32)          # a permutation: cycles
        p[1, K // 2] = K + 5                                           # outside: stays
    eff = torch.where((p < 0) | (p >= K), torch.arange(K, dtype=torch.int32), p).long()
    ref = torch.stack([x[:, b][:, eff[b]] for b in range(B)], dim=1)
    xd = x.to(cuda_device)
    out = None if in_place else torch.full_like(xd, 7)
    got = wkv7.beam_reorder(p.to(cuda_device), xd, batch_dim=1, out=out)
    assert torch.equal(got.cpu(), ref)
    assert torch.equal(xd.cpu(), ref if in_place else x)


def test_reorder_past_32_bit_offsets(cuda_device):
    L, B, K = 9, 2, 4
    row = (1 << 26) + 16                               # 4.8 GB in all
    if torch.cuda.mem_get_info()[0] < 20e9:
        pytest.skip("needs 20 GB")
    x = torch.zeros(L, B, K, row, dtype=torch.uint8, device=cuda_device)
    x[-1, -1] = torch.arange(1, K + 1, device=cuda_device, dtype=torch.uint8)[:, None]
    p = torch.tensor([[0, 1, 2, 3], [1, 0, 3, 3]], dtype=torch.int32, device=cuda_device)
    wkv7.beam_reorder(p, x, batch_dim=1)
    for j, v in enumerate((2, 1, 4, 4)):
        assert bool(torch.all(x[-1, -1, j] == v))
    assert bool(torch.all(x[:, 0] == 0))


def test_decoding_loop(cuda_device):
    """Prefill a prompt per request, then beam search with the states advanced in a pool and moved
    to the picked beams, against the same loop in the oracle."""
    B, K, H, N, V, steps = 2, 3, 2, 64, 301, 6
    g = torch.Generator().manual_seed(44)
    tables = {n: (torch.randn(V, s, generator=g) * c).bfloat16()
              for n, s, c in (("q", H * N, 1.0), ("k", H * N, 1.0), ("v", H * N, 1.0))}
    gate = (-torch.nn.functional.softplus(torch.randn(V, H, generator=g))).bfloat16()
    beta = torch.sigmoid(torch.randn(V, H, generator=g)).bfloat16()
    head = (torch.randn(H * N, V, generator=g) * 0.4).double()
    prompt = torch.randint(0, V, (B, 37), generator=g)

    def tok(t, dev):
        lead = tuple(t.shape)
        d = [tables[n][t].reshape(*lead, H, N) for n in "qkv"] + [gate[t], beta[t]]
        return [x.to(dev) for x in d]

    _, S = wkv7.delta_forward(*tok(prompt, cuda_device), qk_norm=True)
    _, Sr = delta.delta_recurrence(*tok(prompt, "cpu"), qk_norm=True)
    pool = S.repeat_interleave(K, 0).contiguous()
    ref = np.repeat(Sr, K, 0)
    scores = torch.full((B, K), float("-inf"))
    scores[:, 0] = 0.0
    rs, scores = scores.double().numpy(), scores.to(cuda_device)
    ended, rend = torch.zeros(B, K, dtype=torch.bool, device=cuda_device), np.zeros((B, K), bool)
    last = prompt[:, -1:].repeat(1, K)
    for _ in range(steps):
        y = wkv7.delta_step(*tok(last.reshape(-1), cuda_device), pool, qk_norm=True)
        yr, ref = delta.delta_recurrence(*(x[:, None] for x in tok(last.reshape(-1), "cpu")), ref, qk_norm=True)
        assert y_err(y[:, None], yr) <= Y_TOL["bf16"] and s_err(pool, ref) <= 1e-5
        # one set of logits for both loops, so that a rounding does not decide a pick
        logits = (torch.tensor(yr).reshape(B, K, H * N) @ head).float()
        scores, parents, tokens = wkv7.beam_select(logits.to(cuda_device), scores, K, finished=ended, eos=1)
        rs, rp, rt = delta.beam_select(logits.double().numpy(), rs, K, rend, eos=1)
        assert np.array_equal(parents.cpu().numpy(), rp) and np.array_equal(tokens.cpu().numpy(), rt)
        wkv7.beam_reorder(parents, pool.view(B, K, H, N, N))
        ref = ref.reshape(B, K, H, N, N)[np.arange(B)[:, None], rp].reshape(B * K, H, N, N)
        ended = torch.gather(ended, 1, parents.long()) | (tokens == 1)
        rend = np.take_along_axis(rend, rp, 1) | (rt == 1)
        last = tokens.cpu().long()
    assert np.max(np.abs(scores.cpu().numpy() - rs)) <= 1e-5 * np.max(np.abs(rs))


def test_select_and_reorder_in_one_graph_on_another_stream(cuda_device):
    """Captured together on a stream of the caller's and replayed with other logits."""
    x, s = draw(2, 4, 5001, "bf16", 12)
    x2, s2 = draw(2, 4, 5001, "bf16", 13)
    xd, sd = x.to(cuda_device), s.to(cuda_device)
    st = torch.randn(3, 2, 4, 512, device=cuda_device)
    first = st.clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        wkv7.beam_select(xd, sd, 4)                   # attributes are raised before the capture
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = wkv7.beam_select(xd, sd, 4)
            wkv7.beam_reorder(out[1], st, batch_dim=1)
        st.copy_(first)
        xd.copy_(x2)
        sd.copy_(s2)
        graph.replay()
    stream.synchronize()
    ref = delta.beam_select(x2.double().numpy(), s2.numpy(), 4)
    assert np.array_equal(out[1].cpu().numpy(), ref[1]) and np.array_equal(out[2].cpu().numpy(), ref[2])
    p = out[1].long()
    assert torch.equal(st, first[:, torch.arange(2, device=cuda_device)[:, None], p])


def test_two_selections_at_once(cuda_device):
    """On two streams, each with its own workspace, many times over: the same as one after the other."""
    cases = [draw(8, 8, 30_001, "bf16", 91), draw(6, 5, 20_000, "f32", 92)]
    cases = [(x.to(cuda_device), s.to(cuda_device)) for x, s in cases]
    ref = [wkv7.beam_select(x, s, 10) for x, s in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        got = [wkv7.beam_select(x, s, 10, stream=t) for (x, s), t in zip(cases, streams)]
    torch.cuda.synchronize()
    for g, r in zip(got, ref):
        assert all(torch.equal(a, b) for a, b in zip(g, r))
