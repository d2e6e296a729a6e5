"""What the gated-delta-rule and beam operators of this library are measured on.

The operators, with S a head's [N][N] state (row = value channel, column = key channel), q and k
optionally brought to unit length, q scaled, and the gates g (log decay) and beta per token and head:

    e_t = v_t - exp(g_t) S_{t-1} k_t,   S_t = exp(g_t) S_{t-1} + beta_t e_t k_t^T,   y_t = S_t q_t

``forward`` runs it over whole sequences (a batch of equal lengths, or packed ragged ones),
``backward`` gives the gradients of all its inputs, ``step`` advances one token per live row of a
pool of states. ``select`` picks the best continuations over beams and vocabulary, ``reorder``
moves the rows of recurrent states to the beams that were picked.

``run`` computes them in their plain form, or through the library's entry points where ``own`` is set.
"""
import math
import random

import torch

own = False

C = 64          # tokens per chunk of the plain form
EPS = 1e-6      # inside the root of the key and query norms
EOS = 2
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases -------------------------------------------------------------------------------------

def _seq(op, name, dt, B, T, H, Hk, N, ragged, state, norm):
    return {"op": op, "name": name, "dt": dt, "B": B, "T": T, "H": H, "Hk": Hk, "N": N, "ragged": ragged,
            "state": state, "norm": norm}


def listed():
    return [
        # the shortest call: one prompt of 64 tokens, two heads, all in fp32 (latency counts)
        _seq("forward", "prefill B1 T64 H2 f32", "f32", 1, 64, 2, 2, 64, False, False, True),
        # a full prefill batch at model width 2048
        _seq("forward", "prefill B16 T4096 H32", "bf16", 16, 4096, 32, 32, 64, False, False, True),
        # one long document: few heads, a long serial chain
        _seq("forward", "prefill B1 T65536 H40", "bf16", 1, 65536, 40, 40, 64, False, False, True),
        # serving: prompts of different lengths packed together, key heads shared by four value heads, states carried in
        _seq("forward", "prefill packed N128", "bf16", 9, 2777, 16, 4, 128, True, True, True),
        # a training step at model width 768, keys and queries normalised beforehand
        _seq("backward", "backward B8 T1024 H12", "bf16", 8, 1024, 12, 12, 64, False, False, False),
        # training on packed documents, head size 128, shared key heads, with the states' gradients
        _seq("backward", "backward packed N128", "bf16", 7, 1999, 8, 4, 128, True, True, True),
        # one user's next token (latency counts)
        {"op": "step", "name": "step B1 H40", "dt": "bf16", "B": 1, "H": 40, "Hk": 40, "N": 64, "live": 1, "pool": 1,
         "norm": True},
        # a serving batch padded to 256 rows, its states scattered over a larger pool
        {"op": "step", "name": "step B256 H40 pool", "dt": "bf16", "B": 256, "H": 40, "Hk": 40, "N": 64, "live": 250,
         "pool": 320, "norm": True},
        # one request with four beams
        {"op": "select", "name": "select B1 K4", "dt": "f32", "B": 1, "K": 4, "V": 65536, "M": 8, "finished": False},
        # a batch of requests with eight beams each, some of which have ended; an odd vocabulary
        {"op": "select", "name": "select B64 K8", "dt": "bf16", "B": 64, "K": 8, "V": 50277, "M": 16, "finished": True},
        # one request's states: 24 layers of 12 heads
        {"op": "reorder", "name": "reorder B1 K4 L24", "L": 24, "B": 1, "K": 4, "H": 12, "N": 64, "sources": 2},
        # a batch of them, half of the beams replaced
        {"op": "reorder", "name": "reorder B16 K8 L24", "L": 24, "B": 16, "K": 8, "H": 12, "N": 64, "sources": 5},
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["forward", "forward", "backward", "backward", "step", "select", "reorder"])
    if op in ("forward", "backward"):
        N = rng.choice([64, 128])
        H = rng.randint(1, 40)
        Hk = rng.choice([h for h in range(1, H + 1) if H % h == 0])
        ragged = rng.random() < 0.5
        dt = rng.choice(["bf16", "bf16", "f32"])
        cap = (2_000_000 if op == "forward" else 100_000) // (N // 64) ** 2 // (1 if dt == "bf16" else 4)   # token-heads
        T = _logint(rng, 1, 60_000 if op == "forward" and not ragged else 4000)
        T = max(1, min(T, cap // H))
        B = max(1, min(_logint(rng, 1, 24), cap // (H * T)))
        return {"op": op, "dt": dt, "B": B, "T": T, "H": H, "Hk": Hk, "N": N,
                "ragged": ragged, "state": rng.random() < 0.5, "norm": rng.random() < 0.7}
    if op == "step":
        N, B, H = rng.choice([64, 128]), _logint(rng, 1, 256), rng.randint(1, 40)
        Hk = rng.choice([h for h in range(1, H + 1) if H % h == 0])
        if N == 128:
            B = max(1, B // 4)
        live = rng.randint(max(1, B // 2), B)
        return {"op": op, "dt": rng.choice(["bf16", "f32"]), "B": B, "H": H, "Hk": Hk, "N": N, "live": live,
                "pool": B + rng.randint(0, 64), "norm": rng.random() < 0.7}
    if op == "select":
        K = rng.randint(1, 16)
        V = _logint(rng, 1000, 200_000)
        B = max(1, min(_logint(rng, 1, 64), 25_000_000 // (K * V)))
        return {"op": op, "dt": rng.choice(["bf16", "f32"]), "B": B, "K": K, "V": V, "M": rng.randint(1, 2 * K),
                "finished": rng.random() < 0.5}
    K = rng.randint(2, 16)
    N, H, L = rng.choice([64, 128]), rng.randint(1, 32), rng.randint(1, 24)
    B = max(1, min(_logint(rng, 1, 16), 600_000_000 // (L * K * H * N * N * 4)))
    L = max(1, min(L, 600_000_000 // (B * K * H * N * N * 4)))
    return {"op": op, "L": L, "B": B, "K": K, "H": H, "N": N, "sources": rng.randint(1, K - 1)}


def _lens(case):
    """Lengths of the sequences: all T, or ragged from one token (or none) to T."""
    B, T = case["B"], case["T"]
    if not case["ragged"]:
        return [T] * B
    r = random.Random(B * 1_000_003 + T)
    lens = [r.randint(1, T) for _ in range(B)]
    lens[0] = T
    if B > 2:
        lens[1] = 1
    if B > 3:
        lens[2] = 0
    return lens


# ---- inputs ------------------------------------------------------------------------------------

def _gates(gen, dev, shape):
    """Log decays as a trained gate gives them (a rate per head times a softplus of the token's value,
    from almost none to e^-2 or so a token), and write strengths in (0, 1)."""
    H = shape[-1]
    rate = torch.empty(H, device=dev).uniform_(1.0, 16.0, generator=gen)
    bias = torch.empty(H, device=dev).uniform_(math.log(1e-3), math.log(0.1), generator=gen)
    z = torch.randn(shape, device=dev, generator=gen)
    g = -rate * torch.log1p(torch.exp(0.5 * z + bias))
    beta = torch.sigmoid(torch.randn(shape, device=dev, generator=gen))
    return g, beta


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, device=dev, generator=gen)  # noqa: E731
    st = dict(case)
    op = case["op"]
    if op in ("forward", "backward", "step"):
        dt, N, H, Hk = DT[case["dt"]], case["N"], case["H"], case["Hk"]
        st["scale"] = N ** -0.5
        if op == "step":
            lead = (case["B"],)
        else:
            lens = _lens(case)
            cu = [0]
            for n in lens:
                cu.append(cu[-1] + n)
            st["lens"], st["cu"] = lens, torch.tensor(cu, dtype=torch.int32, device=dev)
            lead = (cu[-1],) if case["ragged"] else (case["B"], case["T"])
        q, k, v = rnd(*lead, Hk, N), rnd(*lead, Hk, N), rnd(*lead, H, N)
        if not case["norm"]:
            q, k = (x / x.square().sum(-1, keepdim=True).sqrt() for x in (q, k))
        g, beta = _gates(gen, dev, (*lead, H))
        st.update(q=q.to(dt), k=k.to(dt), v=v.to(dt), g=g.to(dt), beta=beta.to(dt))
        if op == "step":
            st["S"] = 0.1 * rnd(case["pool"], H, N, N)
            slots = torch.full((case["B"],), -1, dtype=torch.int32, device=dev)
            slots[:case["live"]] = torch.randperm(case["pool"], device=dev, generator=gen)[:case["live"]].to(torch.int32)
            st["slots"] = slots
        else:
            st["S0"] = 0.1 * rnd(case["B"], H, N, N) if case["state"] else None
        if op == "backward":
            st["dy"] = rnd(*lead, H, N).to(dt)
            st["dS_T"] = 0.1 * rnd(case["B"], H, N, N) if case["state"] else None
    elif op == "select":
        B, K, V = case["B"], case["K"], case["V"]
        st["logits"] = (2.5 * rnd(B, K, V)).to(DT[case["dt"]])
        st["scores"] = -20.0 + 2.0 * rnd(B, K)
        st["ended"] = (torch.rand(B, K, device=dev, generator=gen) < 0.2) if case["finished"] else None
    else:
        L, B, K, H, N, s = (case[n] for n in ("L", "B", "K", "H", "N", "sources"))
        st["S"] = rnd(L, B, K, H, N, N)
        # s beams survive (the first two of them trade places when there are two), the others take a survivor's state
        order = torch.argsort(torch.rand(B, K, device=dev, generator=gen), dim=1)
        origin = torch.arange(K, device=dev)
        origin = torch.where(origin < s, origin, (origin - s) % s)
        if s >= 2:
            origin[0], origin[1] = 1, 0
        parents = torch.empty(B, K, dtype=torch.int64, device=dev)
        parents.scatter_(1, order, order[:, origin])
        st["parents"] = parents.to(torch.int32)
    return st


def work(case):
    op = case["op"]
    if op in ("forward", "backward", "step"):
        N, H, Hk = case["N"], case["H"], case["Hk"]
        e = 2 if case["dt"] == "bf16" else 4
        tokens = case["live"] if op == "step" else sum(_lens(case))
        rows = case["live"] if op == "step" else case["B"]
        tok = tokens * e * (2 * Hk * N + 2 * H * N + 2 * H)      # q, k, v, the gates, and y (or dy)
        states = rows * H * N * N * 4
        if op == "forward":
            return {"bytes": tok + states * (2 if case["state"] else 1), "flops": tokens * H * 7 * N * N}
        if op == "backward":   # the gradients of q, k, v and the gates too; S0 and dS_T in, dS0 out
            return {"bytes": tok + tokens * e * (2 * Hk * N + H * N + 2 * H) + (3 * states if case["state"] else 0),
                    "flops": tokens * H * 23 * N * N}
        return {"bytes": tok + 2 * states + 4 * case["B"], "flops": tokens * H * 7 * N * N}
    if op == "select":
        B, K, V, M = case["B"], case["K"], case["V"], case["M"]
        return {"bytes": B * K * V * (2 if case["dt"] == "bf16" else 4) + B * K * 5 + B * M * 12, "flops": 4 * B * K * V}
    K, s = case["K"], case["sources"]
    written = K - s + (2 if s >= 2 else 0)
    read = max(min(s, K - s), 2 if s >= 2 else 1)
    return {"bytes": case["L"] * case["B"] * (written + read) * case["H"] * case["N"] ** 2 * 4 + 4 * case["B"] * K,
            "flops": 0}


# ---- plain forms -------------------------------------------------------------------------------

def _pad(st):
    """Indexes of the tokens laid out as [sequence][whole chunks], and which of the places hold one."""
    longest = max(st["lens"])
    L = max(C, -(-longest // C) * C)
    cu = st["cu"].long()
    at = torch.arange(L, device=cu.device)
    live = at < (cu[1:] - cu[:-1])[:, None]
    return torch.where(live, cu[:-1, None] + at, 0), live


def _laid(x, idx, live):
    """[tokens][heads](...) -> fp32 [sequence][heads][chunk][token](...), zeros where there is no token."""
    y = x[idx].float()
    y = y * live.reshape(live.shape + (1,) * (y.dim() - 2)) if y.dim() > 2 else y * live
    S, L = live.shape
    return y.reshape(S, L // C, C, *y.shape[2:]).movedim(3, 1)


def _flat(st, name):
    x = st[name]
    return x if st["ragged"] else x.reshape(-1, *x.shape[2:])


def _unit(x, norm):
    return x * torch.rsqrt(x.square().sum(-1, keepdim=True) + EPS) if norm else x


def _local(st):
    """What the chunks have apart from the state: the inputs laid out, the decays, M_ij = D_ij k_i k_j,
    P_ij = D_ij q_i k_j and the inverse of I + M diag(beta)."""
    idx, live = _pad(st)
    q, k, v, g, b = (_laid(_flat(st, n), idx, live) for n in ("q", "k", "v", "g", "beta"))
    rep = st["H"] // st["Hk"]
    q, k = (_unit(x, st["norm"]).repeat_interleave(rep, dim=1) for x in (q, k))
    q = q * st["scale"]
    G = g.double().cumsum(-1)
    low = torch.ones(C, C, dtype=torch.bool, device=q.device).tril()
    D = torch.where(low, torch.exp(G[..., :, None] - G[..., None, :]), 0).float()
    M = D.tril(-1) * (k @ k.mT)
    A = M * b[..., None, :]
    inv = torch.eye(C, device=q.device).expand_as(A).contiguous()
    for i in range(1, C):
        inv[..., i, :i] = -(A[..., i:i + 1, :i] @ inv[..., :i, :i])[..., 0, :]
    P = D * (q @ k.mT)
    into = torch.exp(G).float()                          # from the chunk's start to each token
    out = torch.exp(G[..., -1:] - G).float()             # from each token to the chunk's end
    return idx, live, q, k, v, b, D, M, P, inv, into, out


def _start(st, like):
    B, H, N = st["B"], st["H"], st["N"]
    return torch.zeros(B, H, N, N, device=like.device) if st["S0"] is None else st["S0"]


def _back(x, idx, live, n_tokens, dtype):
    """[sequence][heads][chunk][token](...) -> [tokens][heads](...)"""
    x = x.movedim(1, 3)
    x = x.reshape(idx.shape[0], idx.shape[1], *x.shape[3:])
    out = torch.zeros(n_tokens + 1, *x.shape[2:], device=x.device)
    out[torch.where(live, idx, n_tokens)] = x
    return out[:n_tokens].to(dtype)


def _shaped(st, x):
    return x if st["ragged"] else x.reshape(st["B"], st["T"], *x.shape[1:])


def _forward(st):
    idx, live, q, k, v, b, D, M, P, inv, into, out = _local(st)
    S = _start(st, q)
    y = torch.empty_like(v)
    for c in range(v.shape[2]):
        E = inv[:, :, c] @ (v[:, :, c] - into[:, :, c, :, None] * (k[:, :, c] @ S.mT))
        U = b[:, :, c, :, None] * E
        y[:, :, c] = into[:, :, c, :, None] * (q[:, :, c] @ S.mT) + P[:, :, c] @ U
        S = into[:, :, c, -1, None, None] * S + (out[:, :, c, :, None] * U).mT @ k[:, :, c]
    y = _back(y, idx, live, _flat(st, "v").shape[0], st["v"].dtype)
    return {"y": _shaped(st, y), "S_T": S}


def _backward(st):
    idx, live, q, k, v, b, D, M, P, inv, into, out = _local(st)
    S = _start(st, q)
    dy = _laid(_flat(st, "dy"), idx, live)
    n = v.shape[2]
    S_in, E = torch.empty(*v.shape[:3], st["N"], st["N"], device=v.device), torch.empty_like(v)
    for c in range(n):
        S_in[:, :, c] = S
        E[:, :, c] = inv[:, :, c] @ (v[:, :, c] - into[:, :, c, :, None] * (k[:, :, c] @ S.mT))
        S = into[:, :, c, -1, None, None] * S + (out[:, :, c, :, None] * b[:, :, c, :, None] * E[:, :, c]).mT @ k[:, :, c]
    dS = torch.zeros_like(S) if st["dS_T"] is None else st["dS_T"]
    dS_out, dX = torch.empty_like(S_in), torch.empty_like(E)
    for c in range(n - 1, -1, -1):
        dS_out[:, :, c] = dS
        dU = P[:, :, c].mT @ dy[:, :, c] + out[:, :, c, :, None] * (k[:, :, c] @ dS.mT)
        dX[:, :, c] = inv[:, :, c].mT @ (b[:, :, c, :, None] * dU)
        w = into[:, :, c, :, None]
        dS = into[:, :, c, -1, None, None] * dS + (w * dy[:, :, c]).mT @ q[:, :, c] - (w * dX[:, :, c]).mT @ k[:, :, c]
    row, col = into[..., None], (out * b)[..., None]
    dP, dM = dy @ E.mT, dX @ E.mT                        # of P and of -M, before beta_j
    pb, mb = D * dP * b[..., None, :], D.tril(-1) * dM * b[..., None, :]
    a_q, a_k, a_o = row * (dy @ S_in), row * (dX @ S_in), E @ dS_out
    dq = a_q + pb @ k
    dk = pb.mT @ q - mb @ k - mb.mT @ k + col * a_o - a_k
    both = P * dP - M * dM
    tail = out * (k * a_o).sum(-1)
    dbeta = both.sum(-2) + tail
    both = both * b[..., None, :]
    dG = both.sum(-1) + (q * a_q).sum(-1) - (k * a_k).sum(-1) - b * dbeta
    last = (b * tail).sum(-1) + into[..., -1] * (S_in * dS_out).sum((-1, -2))
    dg = dG.flip(-1).cumsum(-1).flip(-1) + last[..., None]
    dq = dq * st["scale"]
    rep, dt, count = st["H"] // st["Hk"], st["v"].dtype, _flat(st, "v").shape[0]
    dq, dk = (x.unflatten(1, (st["Hk"], rep)).sum(2) for x in (dq, dk))
    if st["norm"]:
        qr, kr = (_laid(_flat(st, n_), idx, live) for n_ in ("q", "k"))
        dq, dk = _unit_back(qr, dq), _unit_back(kr, dk)
    grads = {"dq": dq, "dk": dk, "dv": dX, "dg": dg, "dbeta": dbeta}
    grads = {n_: _shaped(st, _back(x, idx, live, count, dt)) for n_, x in grads.items()}
    if st["state"]:
        grads["dS0"] = dS
    return grads


def _unit_back(x, dxn):
    r = torch.rsqrt(x.square().sum(-1, keepdim=True) + EPS)
    xn = x * r
    return r * (dxn - xn * (xn * dxn).sum(-1, keepdim=True))


def _step(st):
    live, rep = st["live"], st["H"] // st["Hk"]
    q, k, v, g, b = (st[n][:live].float() for n in ("q", "k", "v", "g", "beta"))
    q, k = (_unit(x, st["norm"]).repeat_interleave(rep, dim=1) for x in (q, k))
    at = st["slots"][:live].long()
    S = torch.exp(g)[..., None, None] * st["S"][at]
    u = b[..., None] * (v - (S @ k[..., None])[..., 0])
    S = S + u[..., :, None] * k[..., None, :]
    st["S"][at] = S
    y = torch.zeros(st["v"].shape, device=v.device)
    y[:live] = (S @ (st["scale"] * q)[..., None])[..., 0]
    return {"y": y.to(st["v"].dtype), "S": st["S"]}


def _select(st):
    x, s, M = st["logits"].double(), st["scores"].double(), st["M"]
    top = x.amax(-1, keepdim=True)
    norm = top + torch.log(torch.exp(x - top).sum(-1, keepdim=True))
    cand = s[..., None] + (x - norm)
    if st["ended"] is not None:
        only = torch.full_like(cand, -math.inf)
        only[..., EOS] = s
        cand = torch.where(st["ended"][..., None], only, cand)
    best, at = torch.sort(cand.flatten(1), dim=1, descending=True, stable=True)
    best, at = best[:, :M], at[:, :M]
    V = st["V"]
    return {"scores": best.float(), "parents": (at // V).int(), "tokens": (at % V).int()}


def _reorder(st):
    S, parents = st["S"], st["parents"].long()
    group = torch.arange(S.shape[1], device=S.device)[:, None]
    S.copy_(S[:, group, parents])
    return S


# ---- the library's entry points ----------------------------------------------------------------

def _own(st):
    from linear_rnn_sequence_rwkv_b200 import wkv7
    op = st["op"]
    if op == "select":
        s, p, t = wkv7.beam_select(st["logits"], st["scores"], st["M"], finished=st["ended"], eos=EOS)
        return {"scores": s, "parents": p, "tokens": t}
    if op == "reorder":
        return wkv7.beam_reorder(st["parents"], st["S"], batch_dim=1)
    x = tuple(st[n] for n in ("q", "k", "v", "g", "beta"))
    kw = {"scale": st["scale"], "qk_norm": st["norm"], "norm_eps": EPS}
    if op == "step":
        y = wkv7.delta_step(*x, st["S"], slots=st["slots"], **kw)
        return {"y": y, "S": st["S"]}
    if st["ragged"]:
        kw["cu_seqlens"] = st["cu"]
    if op == "forward":
        y, S = wkv7.delta_forward(*x, st["S0"], **kw)
        return {"y": y, "S_T": S}
    out = wkv7.delta_backward(*x, st["dy"], st["S0"], st["dS_T"], return_state_grad=st["state"], **kw)
    return {n: t for n, t in out.items() if t is not None}


def run(state):
    if own:
        return _own(state)
    return {"forward": _forward, "backward": _backward, "step": _step, "select": _select,
            "reorder": _reorder}[state["op"]](state)


# ---- the definitions in 64 bits, token by token ------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "reorder":
        S = st["S"].double()
        flat, p = S.flatten(3), st["parents"].long()
        return torch.gather(flat, 2, p[None, :, :, None].expand(flat.shape)).reshape(S.shape)
    if op == "select":
        logp = torch.log_softmax(st["logits"].double(), dim=-1) + st["scores"].double()[..., None]
        if st["ended"] is not None:
            logp = logp.masked_fill(st["ended"][..., None], -math.inf)
            logp[..., EOS] = torch.where(st["ended"], st["scores"].double(), logp[..., EOS])
        return {"scores": logp.flatten(1).topk(case["M"], dim=1).values, "parents": None, "tokens": None}
    rep = case["H"] // case["Hk"]
    raw = {n: st[n].double() for n in ("q", "k", "v", "g", "beta")}
    unit = lambda x: x / (x.square().sum(-1, keepdim=True) + EPS).sqrt() if case["norm"] else x  # noqa: E731
    q = unit(raw["q"]).repeat_interleave(rep, -2) * st["scale"]
    k = unit(raw["k"]).repeat_interleave(rep, -2)
    v, decay, beta = raw["v"], raw["g"].exp(), raw["beta"]
    if op == "step":
        n = case["live"]
        S = st["S"].double()
        y = torch.zeros_like(v)
        at = st["slots"][:n].long()
        old = decay[:n, :, None, None] * S[at]
        new = old + torch.einsum("bhi,bhj->bhij", beta[:n, :, None] * (v[:n] - torch.einsum("bhij,bhj->bhi", old, k[:n])), k[:n])
        S[at] = new
        y[:n] = torch.einsum("bhij,bhj->bhi", new, q[:n])
        return {"y": y, "S": S}
    # one group of sequences at a time: all of them where they are equally long
    if case["ragged"]:
        cu = st["cu"].tolist()
        groups = [(slice(a, b), slice(i, i + 1)) for i, (a, b) in enumerate(zip(cu[:-1], cu[1:]))]
        pick = lambda x, s: x[s][None]  # noqa: E731
    else:
        groups = [(slice(None), slice(None))]
        pick = lambda x, s: x  # noqa: E731
    fn = _exact_backward if op == "backward" else _exact_forward
    parts = []
    for s, b in groups:
        S = torch.zeros(case["B"], case["H"], case["N"], case["N"], device=v.device, dtype=torch.float64)[b] \
            if st["S0"] is None else st["S0"][b].double()
        extra = {}
        if op == "backward":
            extra = {"dy": pick(st["dy"].double(), s), "dS": torch.zeros_like(S) if st["dS_T"] is None else st["dS_T"][b].double()}
        parts.append(fn(*(pick(x, s) for x in (q, k, v, decay, beta)), S, **extra))
    out = {}
    for n in parts[0]:
        state = n in ("S_T", "dS0")
        out[n] = torch.cat([p[n] if state or not case["ragged"] else p[n][0] for p in parts])
    if op == "backward":
        for n, r in (("dq", raw["q"]), ("dk", raw["k"])):
            x = out[n].unflatten(-2, (case["Hk"], rep)).sum(-2)
            if n == "dq":
                x = x * st["scale"]
            if case["norm"]:
                r2 = r.square().sum(-1, keepdim=True) + EPS
                x = x / r2.sqrt() - r * (r * x).sum(-1, keepdim=True) / r2 ** 1.5
            out[n] = x
        if not case["state"]:
            del out["dS0"]
    return out


def _exact_forward(q, k, v, decay, beta, S):
    y = torch.zeros_like(v)
    for t in range(v.shape[1]):
        S = S * decay[:, t, :, None, None]
        kt = k[:, t, :, :, None]
        u = beta[:, t, :, None, None] * (v[:, t, :, :, None] - S @ kt)
        S = S + u * kt.mT
        y[:, t] = (S @ q[:, t, :, :, None])[..., 0]
    return {"y": y, "S_T": S}


def _exact_backward(q, k, v, decay, beta, S, dy, dS):
    T = v.shape[1]
    kept, errs = [], []
    for t in range(T):
        kept.append(S)
        P = S * decay[:, t, :, None, None]
        e = v[:, t] - (P @ k[:, t, :, :, None])[..., 0]
        errs.append(e)
        S = P + (beta[:, t, :, None] * e)[..., :, None] * k[:, t, :, None, :]
    dq, dk, dv, dg, db = (torch.zeros_like(x) for x in (q, k, v, decay, beta))
    for t in range(T - 1, -1, -1):
        a, b, kt, e = decay[:, t, :, None, None], beta[:, t, :, None], k[:, t], errs[t]
        P = kept[t] * a
        St = P + (b * e)[..., :, None] * kt[..., None, :]
        dyt = dy[:, t]
        dS = dS + dyt[..., :, None] * q[:, t, :, None, :]
        dq[:, t] = (St.mT @ dyt[..., None])[..., 0]
        du = (dS @ kt[..., None])[..., 0]
        de = b * du
        dP = dS - de[..., :, None] * kt[..., None, :]
        dk[:, t] = (dS.mT @ (b * e)[..., None])[..., 0] - (P.mT @ de[..., None])[..., 0]
        dv[:, t] = de
        db[:, t] = (du * e).sum(-1)
        dg[:, t] = (dP * P).sum((-1, -2))
        dS = dP * a
    # q carries its scale here, so the gradient is that of the scaled query
    return {"dq": dq, "dk": dk, "dv": dv, "dg": dg, "dbeta": db, "dS0": dS}
