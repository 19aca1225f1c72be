"""A dense product with its epilogue, float64: the router's projection, shared
experts and projections added to the routed layer's output.

    out = act(x w^T + b) + r,   gated: out = act(x wg^T + bg) (x wu^T + bu) + r

with wg the first half of w's rows and wu the second. FFN form as in ``ffn``
(SwiGLU: the gate's activation is silu). No intermediate rounding.
"""
from __future__ import annotations

import math

import numpy as np

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def activate(v: np.ndarray, act: str) -> np.ndarray:
    with np.errstate(over="ignore"):
        if act == "relu":
            return np.where(v < 0.0, 0.0, v)
        if act == "silu":
            return v / (1.0 + np.exp(-v))
        if act == "gelu":
            return 0.5 * v * _erfc(-v / math.sqrt(2.0))  # 1 + erf would cancel far below 0
        if act == "gelu_tanh":
            # (1 + tanh z) / 2 = 1 / (1 + e^-2z), which does not cancel
            return v / (1.0 + np.exp(-math.sqrt(8.0 / math.pi) * (v + 0.044715 * v ** 3)))
    assert act == "none", act
    return v


def preactivation(x, w, bias=None) -> np.ndarray:
    v = np.asarray(x, dtype=np.float64) @ np.asarray(w, dtype=np.float64).T
    return v if bias is None else v + np.asarray(bias, dtype=np.float64)


def linear(x, w, bias=None, act: str = "none", gated: bool = False, residual=None) -> np.ndarray:
    v = preactivation(x, w, bias)
    if gated:
        n = v.shape[1] // 2
        v = activate(v[:, :n], act) * v[:, n:]
    else:
        v = activate(v, act)
    return v if residual is None else v + np.asarray(residual, dtype=np.float64)
