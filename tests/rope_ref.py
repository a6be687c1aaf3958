"""Plain restatement (numpy) of the position rotation for the tests: one pair at a
time, in the roundings that are asked for."""
import numpy as np


def columns(D, rot, pairs):
    """Columns of the first and the second value of each pair."""
    i = np.arange(rot // 2)
    return (i, i + rot // 2) if pairs == "half" else (2 * i, 2 * i + 1)


def angles(n, rot, base=10000.0):
    """float32 tables [n, rot / 2], computed in 64 bits."""
    f = base ** (-np.arange(rot // 2) / max(1, rot // 2))
    a = np.arange(n)[:, None] * f
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def rotate(x, cos, sin, pos, pairs, inverse=False, dtype=np.float64):
    """x [rows, H, D] turned by the angles of pos [rows], every operation in `dtype`;
    NaN where the position is not in the table."""
    y = x.astype(dtype).copy()
    a, b = columns(x.shape[-1], 2 * cos.shape[1], pairs)
    for r in range(x.shape[0]):
        if not 0 <= pos[r] < cos.shape[0]:
            y[r][:, np.concatenate([a, b])] = np.nan
            continue
        c, s = cos[pos[r]].astype(dtype), sin[pos[r]].astype(dtype)
        s = -s if inverse else s
        x1, x2 = x[r][:, a].astype(dtype), x[r][:, b].astype(dtype)
        y[r][:, a] = x1 * c - x2 * s
        y[r][:, b] = x2 * c + x1 * s
    return y
