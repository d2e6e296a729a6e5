"""Row strides whose reach does not fit 64 bits are refused by the library (CPU)."""
import ctypes

import pytest

from linear_rnn_sequence_rwkv_b200 import build, wkv7

BASE, STEP = 1 << 40, 1 << 44       # buffers far enough apart for what the sizes below need
WIDE = 1 << 40                      # the widest stride that is taken: 2^23 rows of bf16 reach over 2^64 bytes


@pytest.fixture(scope="module")
def lib():
    build.build()
    return wkv7.load()


def _ptrs(n):
    return [ctypes.c_void_p(BASE + i * STEP) for i in range(n)]


def _opts(name):
    o = wkv7.DeltaOpts()
    wkv7.load().wkv7_delta_opts_default(ctypes.byref(o))
    setattr(o, name, WIDE)
    return ctypes.byref(o)


@pytest.mark.parametrize("name", ["q_stride", "k_stride", "v_stride"])
def test_delta_strides(lib, name):
    rows = (1 << 23) + 1
    p = _ptrs(15)
    assert lib.wkv7_delta_forward(1, rows, 1, 1, 64, wkv7.BF16, *p[:8], _opts(name), None) == wkv7.ERR_ARG
    assert b"overflow" in lib.wkv7_last_error()
    assert lib.wkv7_delta_backward(1, rows, 1, 1, 64, wkv7.BF16, *p[:14], _opts(name), p[14], 1 << 43, None) == wkv7.ERR_ARG
    assert b"overflow" in lib.wkv7_last_error()
    assert lib.wkv7_delta_step(rows, 1, 1, 64, wkv7.BF16, *p[:6], rows, *p[6:8], _opts(name), None) == wkv7.ERR_ARG
    assert b"overflow" in lib.wkv7_last_error()


def test_logits_stride(lib):
    p = _ptrs(7)
    assert lib.wkv7_beam_select((1 << 23) + 1, 1, 100, 2, wkv7.BF16, p[0], WIDE, p[1], p[2], 0, *p[3:], 1 << 40,
                                None) == wkv7.ERR_ARG
    assert b"overflow" in lib.wkv7_last_error()


@pytest.mark.parametrize("dt,off", [(wkv7.F32, 1), (wkv7.F32, 2), (wkv7.BF16, 1), (wkv7.BF16, 3)])
def test_logits_are_aligned_to_their_elements(lib, dt, off):
    p = _ptrs(7)
    assert lib.wkv7_beam_select(1, 2, 100, 2, dt, ctypes.c_void_p(BASE + off), 0, p[1], p[2], 0, *p[3:], 1 << 20, None) == wkv7.ERR_ALIGN
    assert b"logits" in lib.wkv7_last_error()


@pytest.mark.parametrize("dt,off", [(wkv7.F32, 4), (wkv7.BF16, 2)])
def test_logits_that_start_anywhere_may_not_overlap_outputs(lib, dt, off):
    p = _ptrs(7)
    at = ctypes.c_void_p(p[3].value - off)
    assert lib.wkv7_beam_select(1, 2, 100, 2, dt, at, 0, p[1], p[2], 0, *p[3:], 1 << 20, None) == wkv7.ERR_ARG
    assert b"overlaps" in lib.wkv7_last_error()
