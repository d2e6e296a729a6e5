"""Refusals of the gated-delta and beam entries, on the host before anything is enqueued (CPU)."""
import ctypes

import pytest
import torch

from linear_rnn_sequence_rwkv_b200 import build, wkv7

BASE = 0x10000
STEP = 1 << 26


@pytest.fixture(scope="module")
def lib():
    build.build()
    return wkv7.load()


def _opts(**kw):
    o = wkv7.DeltaOpts()
    wkv7.load().wkv7_delta_opts_default(ctypes.byref(o))
    for n, v in kw.items():
        setattr(o, n, v)
    return o


def _ptrs(names, over):
    base = {n: BASE + (i + 1) * STEP for i, n in enumerate(names)}
    base.update(over or {})
    return [None if base[n] is None else ctypes.c_void_p(base[n]) for n in names]


def _fwd(lib, ptrs=None, B=1, T=4, H=2, Hk=1, N=64, dt=1, **opts):
    p = _ptrs(("q", "k", "v", "g", "beta", "S0", "y", "S_T"), ptrs)
    return lib.wkv7_delta_forward(B, T, H, Hk, N, dt, *p, ctypes.byref(_opts(**opts)), None)


def _bwd(lib, ptrs=None, B=1, T=4, H=2, Hk=1, N=64, dt=1, ws_bytes=1 << 22, **opts):
    p = _ptrs(("q", "k", "v", "g", "beta", "S0", "dy", "dS_T", "dq", "dk", "dv", "dg", "dbeta", "dS0", "workspace"), ptrs)
    return lib.wkv7_delta_backward(B, T, H, Hk, N, dt, *p[:14], ctypes.byref(_opts(**opts)), p[14], ws_bytes, None)


def _step(lib, ptrs=None, B=1, H=2, Hk=1, N=64, dt=1, n_slots=4, **opts):
    p = _ptrs(("q", "k", "v", "g", "beta", "S", "slots", "y"), ptrs)
    return lib.wkv7_delta_step(B, H, Hk, N, dt, *p[:6], n_slots, *p[6:], ctypes.byref(_opts(**opts)), None)


def _select(lib, ptrs=None, B=1, K=2, V=100, M=2, dt=1, stride=0, eos=0, ws_bytes=1 << 20):
    p = _ptrs(("logits", "scores", "finished", "out_scores", "parents", "tokens", "workspace"), ptrs)
    return lib.wkv7_beam_select(B, K, V, M, dt, p[0], stride, p[1], p[2], eos, *p[3:], ws_bytes, None)


def _reorder(lib, ptrs=None, L=1, B=1, K=2, row=64):
    return lib.wkv7_beam_reorder(L, B, K, row, *_ptrs(("parents", "src", "dst"), ptrs), None)


SIZES = [(dict(B=0), wkv7.ERR_ARG, b"sizes"), (dict(H=0), wkv7.ERR_ARG, b"sizes"), (dict(Hk=0), wkv7.ERR_ARG, b"sizes"),
         (dict(H=3, Hk=2), wkv7.ERR_ARG, b"multiple"), (dict(N=0), wkv7.ERR_ARG, b"sizes"),
         (dict(N=96), wkv7.ERR_UNSUPPORTED, b"head size"), (dict(dt=5), wkv7.ERR_ARG, b"dtype"),
         (dict(scale=float("nan")), wkv7.ERR_ARG, b"scale"), (dict(qk_norm=2), wkv7.ERR_ARG, b"qk_norm"),
         (dict(norm_eps=0.0), wkv7.ERR_ARG, b"norm_eps"), (dict(norm_eps=float("inf")), wkv7.ERR_ARG, b"norm_eps"),
         (dict(q_stride=63), wkv7.ERR_ARG, b"q_stride"), (dict(k_stride=68), wkv7.ERR_ARG, b"k_stride"),
         (dict(v_stride=-128), wkv7.ERR_ARG, b"v_stride"), (dict(B=1 << 30, H=1 << 10), wkv7.ERR_ARG, b"heads"),
         (dict(ptrs={"q": None}), wkv7.ERR_ARG, b"q is NULL"), (dict(ptrs={"beta": None}), wkv7.ERR_ARG, b"beta is NULL"),
         (dict(ptrs={"y": None}), wkv7.ERR_ARG, b"y is NULL"), (dict(ptrs={"k": BASE + 8}), wkv7.ERR_ALIGN, b"k is not"),
         (dict(ptrs={"y": BASE + 3 * STEP}), wkv7.ERR_ARG, b"overlaps")]


@pytest.mark.parametrize("kw,status,word", SIZES)
@pytest.mark.parametrize("entry", [_fwd, _step])
def test_delta_refusals(lib, entry, kw, status, word):
    assert entry(lib, **kw) == status
    assert word in lib.wkv7_last_error()


def test_forward_refusals(lib):
    assert _fwd(lib, T=-1) == wkv7.ERR_ARG
    assert _fwd(lib, T=2147483647, B=1 << 20) == wkv7.ERR_ARG and b"overflow" in lib.wkv7_last_error()
    # S_T may be S0 exactly, not lie across it
    assert _fwd(lib, ptrs={"S_T": BASE + 6 * STEP + 64}) == wkv7.ERR_ARG and b"overlaps" in lib.wkv7_last_error()
    assert _fwd(lib, ptrs={"S_T": BASE + 2 * STEP}) == wkv7.ERR_ARG
    assert _fwd(lib, cu_seqlens=BASE + 4) == wkv7.ERR_ALIGN and b"cu_seqlens" in lib.wkv7_last_error()


@pytest.mark.parametrize("kw,status,word", [c for c in SIZES if "y" not in c[0].get("ptrs", {})])
def test_backward_refusals_as_forward(lib, kw, status, word):
    assert _bwd(lib, **kw) == status
    assert word in lib.wkv7_last_error()


def test_backward_refusals(lib):
    for n in ("dy", "dq", "dk", "dv", "dg", "dbeta"):
        assert _bwd(lib, ptrs={n: None}) == wkv7.ERR_ARG and n.encode() in lib.wkv7_last_error()
    assert _bwd(lib, ws_bytes=16) == wkv7.ERR_WORKSPACE
    assert _bwd(lib, ptrs={"workspace": None}) == wkv7.ERR_WORKSPACE
    assert _bwd(lib, ptrs={"dv": BASE + 7 * STEP}) == wkv7.ERR_ARG and b"overlaps" in lib.wkv7_last_error()   # on dy
    assert _bwd(lib, ptrs={"dS0": BASE + 8 * STEP + 64}) == wkv7.ERR_ARG                                        # across dS_T
    assert _bwd(lib, ptrs={"dbeta": BASE + 15 * STEP}) == wkv7.ERR_ARG                                          # in the workspace
    assert _bwd(lib, T=-1) == wkv7.ERR_ARG


def test_backward_workspace(lib):
    """E in two bf16 terms and dv's second per row and head, two states in two bf16 terms each per chunk
    of 64 (one more per sequence); fp32 keeps E and the states as they are. Where chunks and key heads are
    fewer than the SMs, the value heads of a key head go to several parts, each with dq and dk in fp32."""
    f = lib.wkv7_delta_backward_workspace_bytes
    assert f(2, 100, 4, 2, 64, 1, None) == 3 * 200 * 4 * 64 * 2 + 4 * 5 * 4 * 4096 * 2 + 2 * 2 * 200 * 2 * 64 * 4
    assert f(2, 100, 4, 2, 64, 0, None) == 200 * 4 * 64 * 4 + 2 * 5 * 4 * 4096 * 4 + 2 * 2 * 200 * 2 * 64 * 4
    assert f(2, 100, 4, 4, 64, 1, None) == 3 * 200 * 4 * 64 * 2 + 4 * 5 * 4 * 4096 * 2
    assert f(37, 100, 8, 2, 64, 0, None) == 3700 * 8 * 64 * 4 + 2 * 94 * 8 * 4096 * 4
    o = _opts(cu_seqlens=BASE)
    assert f(3, 100, 4, 2, 128, 1, ctypes.byref(o)) == 3 * 100 * 4 * 128 * 2 + 4 * 4 * 4 * 16384 * 2 + 2 * 2 * 100 * 2 * 128 * 4
    assert f(2, 0, 4, 2, 64, 1, None) == 0 and f(2, 10, 3, 2, 64, 1, None) == 0


def test_step_refusals(lib):
    assert _step(lib, n_slots=0) == wkv7.ERR_ARG and b"n_slots" in lib.wkv7_last_error()
    assert _step(lib, B=5, ptrs={"slots": None}) == wkv7.ERR_ARG and b"without slots" in lib.wkv7_last_error()
    assert _step(lib, cu_seqlens=BASE) == wkv7.ERR_ARG and b"cu_seqlens" in lib.wkv7_last_error()
    assert _step(lib, ptrs={"S": None}) == wkv7.ERR_ARG
    assert _step(lib, n_slots=2147483647, H=1 << 20) == wkv7.ERR_ARG
    assert _step(lib, ptrs={"y": BASE + 6 * STEP}) == wkv7.ERR_ARG and b"overlaps" in lib.wkv7_last_error()


@pytest.mark.parametrize("kw,status,word", [
    (dict(B=0), wkv7.ERR_ARG, b"sizes"), (dict(K=0), wkv7.ERR_ARG, b"sizes"), (dict(V=0), wkv7.ERR_ARG, b"sizes"),
    (dict(M=0), wkv7.ERR_ARG, b"sizes"), (dict(K=65), wkv7.ERR_UNSUPPORTED, b"at most 64"),
    (dict(M=65), wkv7.ERR_UNSUPPORTED, b"at most 64"), (dict(dt=2), wkv7.ERR_ARG, b"dtype"),
    (dict(stride=99), wkv7.ERR_ARG, b"row_stride"), (dict(eos=100), wkv7.ERR_ARG, b"eos"), (dict(eos=-1), wkv7.ERR_ARG, b"eos"),
    (dict(ws_bytes=8), wkv7.ERR_WORKSPACE, b"workspace"), (dict(ptrs={"workspace": None}), wkv7.ERR_WORKSPACE, b"workspace"),
    (dict(ptrs={"logits": None}), wkv7.ERR_ARG, b"logits"), (dict(ptrs={"tokens": None}), wkv7.ERR_ARG, b"tokens"),
    (dict(ptrs={"scores": BASE + 4}), wkv7.ERR_ALIGN, b"scores"),
    (dict(ptrs={"parents": BASE + 6 * STEP}), wkv7.ERR_ARG, b"overlaps"),
    (dict(B=1 << 30, K=64, V=1 << 20), wkv7.ERR_ARG, b"overflow")])
def test_select_refusals(lib, kw, status, word):
    assert _select(lib, **kw) == status
    assert word in lib.wkv7_last_error()


@pytest.mark.parametrize("kw,status,word", [
    (dict(L=0), wkv7.ERR_ARG, b"sizes"), (dict(B=-1), wkv7.ERR_ARG, b"sizes"), (dict(K=0), wkv7.ERR_ARG, b"sizes"),
    (dict(K=65), wkv7.ERR_UNSUPPORTED, b"at most 64"), (dict(row=0), wkv7.ERR_ARG, b"row_bytes"),
    (dict(row=24), wkv7.ERR_ARG, b"row_bytes"), (dict(ptrs={"parents": None}), wkv7.ERR_ARG, b"parents"),
    (dict(ptrs={"src": BASE + 8}), wkv7.ERR_ALIGN, b"src"),
    (dict(ptrs={"dst": BASE + 2 * STEP + 64}), wkv7.ERR_ARG, b"overlaps"),
    (dict(L=1 << 20, B=1 << 20, row=1 << 20), wkv7.ERR_ARG, b"overflow")])
def test_reorder_refusals(lib, kw, status, word):
    assert _reorder(lib, **kw) == status
    assert word in lib.wkv7_last_error()


def test_workspace_query(lib):
    assert lib.wkv7_beam_select_workspace_bytes(0, 1, 1, 1) == 0
    assert lib.wkv7_beam_select_workspace_bytes(1, 65, 10, 1) == 0
    # one segment of 2048: a partial sum of 16 bytes and M keys of 8 per row
    assert lib.wkv7_beam_select_workspace_bytes(2, 3, 100, 5) == 2 * 3 * (16 + 5 * 8)


def _tok(B=2, T=3, H=2, Hk=1, N=64, dtype=torch.bfloat16):
    z = lambda *s: torch.zeros(*s, dtype=dtype)  # noqa: E731
    return [z(B, T, Hk, N), z(B, T, Hk, N), z(B, T, H, N), z(B, T, H), z(B, T, H)]


def test_binding_names_what_is_wrong():
    """Shapes, types and layouts are refused by the binding before the library is called."""
    def bad(i, x, exc=ValueError, **kw):
        t = _tok()
        t[i] = x
        with pytest.raises(exc):
            wkv7.delta_forward(*t, **kw)

    bad(0, torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16))                  # q's heads are not k's
    bad(1, torch.zeros(2, 3, 64, dtype=torch.bfloat16))
    bad(3, torch.zeros(2, 3, 1, dtype=torch.bfloat16))
    bad(3, torch.zeros(2, 3, 2), TypeError)                                 # g of another type
    bad(2, torch.zeros(2, 3, 2, 64, dtype=torch.float16), TypeError)
    bad(2, torch.zeros(2, 3, 64, 2, dtype=torch.bfloat16).mT)               # channels strided
    bad(2, torch.zeros(2, 5, 2, 64, dtype=torch.bfloat16)[:, ::2])          # rows not evenly spaced over the batch
    bad(2, torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16), cu_seqlens=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        wkv7.delta_step(*(x[:, 0] for x in _tok()), torch.zeros(2, 2, 64, 32))
    with pytest.raises(TypeError):
        wkv7.delta_step(*(x[:, 0].contiguous() for x in _tok()), torch.zeros(2, 2, 64, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        wkv7.beam_select(torch.zeros(2, 3), torch.zeros(2, 3), 2)
    with pytest.raises(ValueError):
        wkv7.beam_select(torch.zeros(2, 3, 8), torch.zeros(3, 2), 2)
    with pytest.raises(ValueError):
        wkv7.beam_reorder(torch.zeros(2, 3, dtype=torch.int32), torch.zeros(4, 3, 8))
    with pytest.raises(ValueError):
        wkv7.beam_reorder(torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3, 8, 4).mT)


def test_row_strides_are_recognised():
    wide = torch.zeros(2, 3, 5 * 64, dtype=torch.bfloat16)
    v = wide[..., 64:192].unflatten(-1, (2, 64))
    assert wkv7._row_stride("v", v, (2, 3, 2, 64), torch.bfloat16, v.device) == 320
    assert wkv7._row_stride("v", v[:1, :1], (1, 1, 2, 64), torch.bfloat16, v.device) == 0
