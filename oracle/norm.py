"""Plain CPU reference of the layer norm calls (rs_layer_norm, rs_layer_norm_grad),
from the definitions in 64 bits; the gradients from the chain rule written out."""
from __future__ import annotations

import numpy as np


def _parts(x, eps: float, center: bool):
    x = np.asarray(x, dtype=np.float64)
    dev = x - x.mean(1, keepdims=True) if center else x
    r = 1.0 / np.sqrt((dev * dev).mean(1, keepdims=True) + float(np.float32(eps)))
    return dev * r, r


def norm(x, w, b=None, eps: float = 1e-5, center: bool = True) -> np.ndarray:
    h, _ = _parts(x, eps, center)
    return h * np.asarray(w, dtype=np.float64) + (0.0 if b is None else np.asarray(b, dtype=np.float64))


def norm_grad(x, dy, w, eps: float = 1e-5, center: bool = True):
    """(dx, dw, db) of sum(dy * norm(x, w, b))."""
    dy = np.asarray(dy, dtype=np.float64)
    h, r = _parts(x, eps, center)
    g = dy * np.asarray(w, dtype=np.float64)
    dx = g - h * (g * h).mean(1, keepdims=True)
    if center:
        dx = dx - g.mean(1, keepdims=True)
    return dx * r, (dy * h).sum(0), dy.sum(0)
