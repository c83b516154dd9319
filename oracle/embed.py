"""Plain CPU reference of the embedding calls (rs_embed_rows, rs_embed_grad)."""
from __future__ import annotations

import numpy as np


def lookup(table, ids, scale: float) -> np.ndarray:
    """fl32(scale * table[ids]) in fp32; rows of +0.0 for ids outside the table."""
    table, ids = np.asarray(table, dtype=np.float32), np.asarray(ids)
    named = (ids >= 0) & (ids < table.shape[0])
    out = np.zeros((ids.size, table.shape[1]), dtype=np.float32)
    out[named] = table[ids[named]] * np.float32(scale)
    return out


def sigma(scale: float, inv_v: bool, V: int) -> np.float32:
    return np.float32(np.float64(np.float32(scale)) / V) if inv_v else np.float32(scale)


def row_sums(dy, ids, rows: int):
    """(sum of dy's rows by id, the same of their absolute values, tokens by row) in 64 bits."""
    dy, ids = np.asarray(dy, dtype=np.float64), np.asarray(ids)
    total, size, count = np.zeros((rows, dy.shape[1])), np.zeros((rows, dy.shape[1])), np.zeros(rows, dtype=np.int64)
    for t in np.flatnonzero((ids >= 0) & (ids < rows)):
        total[ids[t]] += dy[t]
        size[ids[t]] += np.abs(dy[t])
        count[ids[t]] += 1
    return total, size, count
