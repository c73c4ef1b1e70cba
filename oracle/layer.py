"""fp64 reference of what stands around the attention in its layer: the residual stream's
addition and RMS norm, and the projections with their epilogue.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py): the library never imports this.

Source. The GatedMLA docs: "Projection geometry and stored weights" (projections stored out
x in, RMS norm), "Output projection and optional gate" (the attention's output times
sigmoid(gate projection of the hidden state), then Wo). The residual's addition before the
norm and after Wo is the usual pre-norm layer's. The 8-bit rows are oracle/fp8.py's.

Everything is float64; nothing is rounded.
"""
from __future__ import annotations

import math

import numpy as np

from . import fp8
from .mla_oracle import rms_norm, to_f64


def add_rmsnorm(x, residual, gain, eps):
    """(s, y): s = x + residual (x alone if None), y = s / sqrt(mean(s^2) + eps) * gain."""
    s = to_f64(x)
    if residual is not None:
        s = s + to_f64(residual)
    return s, rms_norm(s, gain, eps)


def activation(v, act: str):
    v = np.asarray(v, dtype=np.float64)
    if act == "none":
        return v
    with np.errstate(over="ignore"):
        if act == "sigmoid":
            return 1.0 / (1.0 + np.exp(-v))
        if act == "silu":
            return v / (1.0 + np.exp(-v))
    if act == "gelu":
        return 0.5 * v * np.vectorize(math.erfc, otypes=[np.float64])(-v / math.sqrt(2.0))
    raise ValueError(act)


def linear(x, W, bias=None, mul=None, residual=None, act: str = "none"):
    """residual + mul * act(x W^T + bias); x [T, K], W [N, K] out x in."""
    v = to_f64(x) @ to_f64(W).T
    if bias is not None:
        v = v + to_f64(bias)
    v = activation(v, act)
    if mul is not None:
        v = v * to_f64(mul)
    if residual is not None:
        v = v + to_f64(residual)
    return v


def linear_fp8(x_codes, x_scales, W_codes, W_scales, bias=None, mul=None, residual=None, act: str = "none"):
    return linear(fp8.dequantise_rows(x_codes, x_scales), fp8.dequantise_rows(W_codes, W_scales), bias, mul, residual,
                  act)
