"""Inputs and bounds shared by the gated-delta tests.

Bounds (max |got - ref| / max |ref| per sequence and head, as everywhere in these tests):
  * fp32 anywhere, and the fp32 state of bf16 inputs: 1e-5, the bound this library holds fp32 paths to.
    The tensor-core path multiplies operands split into three bf16 terms (24 bits), so it
    stays at fp32's own rounding.
  * bf16 outputs: one rounding of the result (half a step, 2^-8 of the value), and on the
    tensor-core path one rounding each of at most two operands of the sums behind it (2^-8 of
    each term, with signs that vary, so at most about 2^-8 of the largest result each): 3 * 2^-8.
"""
import numpy as np
import torch

from tests.parity_util import as_np, slice_rel_err

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
Y_TOL = {"bf16": 3 * 2.0 ** -8, "f32": 1e-5}
S_TOL = 1e-5


def make(lead, H, Hk, N, dt, seed, norm=True, gate=1.0):
    """Token tensors on the CPU with the given leading shape, of the given type (values exact in it)."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*lead, *s, generator=g)  # noqa: E731
    d = {"q": r(Hk, N), "k": r(Hk, N), "v": r(H, N), "g": -gate * torch.nn.functional.softplus(r(H) - 2.0),
         "beta": torch.sigmoid(r(H))}
    if not norm:
        for n in "qk":
            d[n] = d[n] / d[n].norm(dim=-1, keepdim=True)
    return {n: x.to(DT[dt]) for n, x in d.items()}


def state(B, H, N, seed):
    return 0.1 * torch.randn(B, H, N, N, generator=torch.Generator().manual_seed(seed))


TOK = ("q", "k", "v", "g", "beta")


def err(got, ref, axes):
    return slice_rel_err(got, ref, axes)


def y_err(got, ref):
    return slice_rel_err(got, ref, (0, 2))


def s_err(got, ref):
    return slice_rel_err(got, ref, (0, 1))


__all__ = ["DT", "Y_TOL", "S_TOL", "TOK", "make", "state", "err", "y_err", "s_err", "as_np", "np"]
