"""Plain CPU reference of the vocabulary head's calls (rs_head_loss, rs_head_grad,
rs_distill_loss, rs_distill_grad), from the definitions in 64 bits."""
from __future__ import annotations

import numpy as np


def shares(ids, rows: int, teacher=None, temperature: float = 1.0):
    """(q per place, whether a token has a target): one-hot for labels, the softmax of the teacher's
    logits over the places that hold a row of the table and are not -inf."""
    ids = np.asarray(ids)
    there = (ids >= 0) & (ids < rows)
    if teacher is None:
        return there.astype(np.float64), there.any(1)
    z = np.where(there, np.asarray(teacher, dtype=np.float64), -np.inf)
    live = (~(z == -np.inf)).any(1)
    q = np.zeros(z.shape)
    with np.errstate(invalid="ignore"):
        e = np.exp((z[live] - z[live].max(1, keepdims=True)) / temperature)
        q[live] = e / e.sum(1, keepdims=True)
    return q, live


def losses(x, table, ids, teacher=None, temperature: float = 1.0, scale: float = 1.0):
    """(loss, softmax p, wanted distribution over the table's rows, whether a token has a target)."""
    x, table, ids = np.asarray(x, dtype=np.float64), np.asarray(table, dtype=np.float64), np.asarray(ids)
    ids = ids.reshape(x.shape[0], -1)
    q, live = shares(ids, table.shape[0], teacher, temperature)
    l = x @ table.T * (float(np.float32(scale)) / temperature)
    top = l.max(1, keepdims=True)
    log_p = l - top - np.log(np.exp(l - top).sum(1, keepdims=True))
    full, loss = np.zeros(l.shape), np.zeros(x.shape[0])
    for t in np.flatnonzero(live):
        for r, s in zip(ids[t], q[t]):
            if 0 <= r < table.shape[0] and s != 0.0:
                full[t, r] += s
                loss[t] += s * (np.log(s) - log_p[t, r])
    return loss * temperature ** 2, np.exp(log_p), full, live


def gradients(x, table, ids, weights, teacher=None, temperature: float = 1.0, scale: float = 1.0):
    """(dx, dtable, and the same two sums over absolute values) of sum weights * losses."""
    x, table = np.asarray(x, dtype=np.float64), np.asarray(table, dtype=np.float64)
    _, p, full, live = losses(x, table, ids, teacher, temperature, scale)
    a = np.where(live, np.asarray(weights, dtype=np.float64) * temperature * float(np.float32(scale)), 0.0)[:, None]
    d, size = a * (p - full), np.abs(a) * np.where(live[:, None], p + full, 0.0)
    return d @ table, d.T @ x, size @ np.abs(table), size.T @ np.abs(x)
