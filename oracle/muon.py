"""Plain CPU reference of the matrix operators (rs_orthogonalize, rs_muon_step):
the Newton-Schulz iteration from its definition, in 64 bits.

The Muon paragraphs of the feynmanwiki walkthrough name the iteration and give
no formula; this is the published quintic: X = G / (|G|_F + eps), then
X <- a X + (b A + c A^2) X with A = X X^T, on G or its transpose, whichever is
wide."""
from __future__ import annotations

import numpy as np

COEFFS = (3.4445, -4.7750, 2.0315)


def is_matrix(spec) -> bool:
    return spec.kind == "WHOLE" and spec.rows > 1 and spec.cols > 1


def orthogonalize(g, coeffs=(COEFFS,) * 5, eps: float = 1e-7) -> np.ndarray:
    g = np.asarray(g, dtype=np.float64)
    x = g.T if g.shape[0] > g.shape[1] else g
    x = x / (np.sqrt((x * x).sum()) + eps)
    for a, b, c in coeffs:
        s = x @ x.T
        x = a * x + (b * s + c * (s @ s)) @ x
    return x.T if g.shape[0] > g.shape[1] else x


def update_scale(mode: str, rows: int, cols: int) -> float:
    return {"none": 1.0, "spectral": max(1.0, rows / cols) ** 0.5, "rms": 0.2 * max(rows, cols) ** 0.5}[mode]


def momentum_f32(mom, grad, mu: float) -> np.ndarray:
    """mu * mom + grad, each operation rounded to fp32."""
    mom, grad, mu = (np.asarray(v, dtype=np.float32) for v in (mom, grad, mu))
    return mu * mom + grad


def muon_direction(mom_new, grad, mu: float, nesterov: bool) -> np.ndarray:
    mom_new, grad, mu = (np.asarray(v, dtype=np.float32) for v in (mom_new, grad, mu))
    return grad + mu * mom_new if nesterov else mom_new
