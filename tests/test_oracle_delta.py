"""The gated-delta and beam oracle against closed forms, another recurrence and differences (CPU)."""
import numpy as np
import pytest

from oracle import delta, reference


def _draw(B, T, H, Hk, N, seed=0, unit=False):
    r = np.random.default_rng(seed)
    q, k, v = r.normal(size=(B, T, Hk, N)), r.normal(size=(B, T, Hk, N)), r.normal(size=(B, T, H, N))
    if unit:
        q, k = (x / np.linalg.norm(x, axis=-1, keepdims=True) for x in (q, k))
    return q, k, v, -np.abs(r.normal(size=(B, T, H))) * 0.3, 1 / (1 + np.exp(-r.normal(size=(B, T, H)))), \
        r.normal(size=(B, H, N, N)) * 0.1


def test_is_wkv7_with_one_decay_for_all_channels():
    """w = exp(g) in every channel, kk the unit key, a = beta exp(g), k = beta times the unit key."""
    q, k, v, g, b, S0 = _draw(2, 9, 3, 3, 8, unit=True)
    w = np.broadcast_to(np.exp(g)[..., None], v.shape)
    a = np.broadcast_to((b * np.exp(g))[..., None], v.shape)
    y, S, _ = reference.wkv7_recurrence(q, w, b[..., None] * k, v, k, a, S0)
    y2, S2 = delta.delta_recurrence(q, k, v, g, b, S0, scale=1.0)
    np.testing.assert_allclose(y2, y, rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(S2, S, rtol=1e-12, atol=1e-13)


def test_closed_forms():
    q, k, v, g, b, S0 = _draw(1, 6, 2, 2, 8, seed=1, unit=True)
    # beta = 1: what was just written is read back whole
    y, _ = delta.delta_recurrence(k, k, v, g, np.ones_like(b), S0, scale=1.0)
    np.testing.assert_allclose(y, v, atol=1e-12)
    # beta = 0: pure decay
    _, S = delta.delta_recurrence(q, k, v, g, np.zeros_like(b), S0)
    np.testing.assert_allclose(S, S0 * np.exp(g.sum(1))[..., None, None], rtol=1e-12)
    # a log decay of -inf forgets everything before it
    g2 = g.copy()
    g2[:, 3] = -np.inf
    y, S = delta.delta_recurrence(q, k, v, g2, b, S0)
    y2, S2 = delta.delta_recurrence(*(x[:, 3:] for x in (q, k, v, g, b)))
    np.testing.assert_allclose(S, S2, atol=1e-13)
    np.testing.assert_allclose(y[:, 3:], y2, atol=1e-13)


@pytest.mark.parametrize("norm,Hk", [(False, 2), (True, 1), (True, 2)])
def test_gradients_against_differences(norm, Hk):
    B, T, H, N = 1, 4, 2, 3
    q, k, v, g, b, S0 = _draw(B, T, H, Hk, N, seed=2)
    r = np.random.default_rng(3)
    dy, dS = r.normal(size=v.shape), r.normal(size=S0.shape)
    args = {"q": q, "k": k, "v": v, "g": g, "beta": b, "S0": S0}
    kw = {"scale": 0.7, "qk_norm": norm, "norm_eps": 1e-2}

    def loss(a):
        y, S = delta.delta_recurrence(*(a[n] for n in ("q", "k", "v", "g", "beta", "S0")), **kw)
        return np.sum(y * dy) + np.sum(S * dS)

    got = delta.delta_backward(q, k, v, g, b, S0, dy, dS, **kw)
    for n, x in args.items():
        for i in r.choice(x.size, size=min(8, x.size), replace=False):
            h = 1e-6
            up, dn = ({**args, n: x.copy()} for _ in range(2))
            up[n].flat[i] += h
            dn[n].flat[i] -= h
            num = (loss(up) - loss(dn)) / (2 * h)
            assert abs(num - got["d" + n].flat[i]) <= 1e-7 * max(1.0, abs(num)), (n, i)


def test_beam_select_by_brute_force():
    r = np.random.default_rng(4)
    x, s = r.normal(size=(3, 2, 11)), r.normal(size=(3, 2))
    x[0, 1, :] = -np.inf
    x[1, 0, 3] = np.nan
    fin = np.zeros((3, 2), bool)
    fin[2, 1] = True
    got_s, got_p, got_t = delta.beam_select(x, s, 5, fin, eos=7)
    for b in range(3):
        every = []
        for j in range(2):
            row = np.where(np.isnan(x[b, j]), -np.inf, x[b, j])
            z = np.exp(row).sum()
            for t in range(11):
                p = np.exp(row[t]) / z if z > 0 else 0.0
                if fin[b, j]:
                    p = 1.0 if t == 7 else 0.0
                if p > 0:
                    every.append((s[b, j] + np.log(p), j, t))
        every.sort(key=lambda c: (-c[0], c[1], c[2]))
        np.testing.assert_allclose(got_s[b], [c[0] for c in every[:5]], rtol=1e-12)
        assert [(p, t) for p, t in zip(got_p[b], got_t[b])] == [c[1:] for c in every[:5]]
    # nothing left to choose
    s2, p2, t2 = delta.beam_select(np.full((1, 1, 4), -np.inf), np.zeros((1, 1)), 2)
    assert np.all(np.isneginf(s2)) and np.all(p2 == -1) and np.all(t2 == -1)
