"""Plain reference of the paged-cache operators, for their tests: NumPy
float32 where the format is defined in float32 (the rotation's products and
sums, scales, quotients, decoded values) and float64 elsewhere.  Packing and
decoding are the oracle's."""

from __future__ import annotations

import numpy as np

import oracle as O


def rope_table(n_pos: int, rot: int, base: float = 10000.0) -> np.ndarray:
    i = np.arange(0, rot, 2, dtype=np.float64)
    a = np.arange(n_pos, dtype=np.float64)[:, None] * base ** (-i / rot)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def pair_index(rot: int, interleaved: bool):
    if interleaved:
        return np.arange(0, rot, 2), np.arange(1, rot, 2)
    return np.arange(rot // 2), np.arange(rot // 2, rot)


def rotate(x: np.ndarray, table, pos, interleaved: bool) -> np.ndarray:
    """x [n, heads, D] turned at positions [n], in x's own precision: float32
    in, every product and sum a float32 one."""
    if table is None:
        return x.copy()
    rot = table.shape[1]
    a, b = pair_index(rot, interleaved)
    c = table[pos][:, None, : rot // 2].astype(x.dtype)
    s = table[pos][:, None, rot // 2:].astype(x.dtype)
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    assert y.dtype == x.dtype
    return y


def norm_rope(x: np.ndarray, w, eps: float, table, pos, interleaved: bool) -> np.ndarray:
    """RMS norm of each head and the rotation in float64."""
    y = x.astype(np.float64)
    if w is not None:
        y = y / np.sqrt(np.mean(y * y, -1, keepdims=True) + eps) * w.astype(np.float64)
    return rotate(y, None if table is None else table.astype(np.float64), pos, interleaved)


def attend_rows(q: np.ndarray, k: np.ndarray, v: np.ndarray, length: int, scale: float, causal: bool) -> np.ndarray:
    """q [n, H_q, D] (the sequence's last n positions), k, v [H_kv, >= length,
    D] decoded values; float64.  A row without a key is zero."""
    n, H_q, D = q.shape
    H = k.shape[0]
    G = H_q // H
    out = np.zeros((n, H_q, D))
    for h in range(H):
        kk, vv = k[h, :length].astype(np.float64), v[h, :length].astype(np.float64)
        s = np.einsum("igd,td->igt", q[:, h * G:(h + 1) * G].astype(np.float64), kk) * scale
        for i in range(n):
            lim = min(length, length - n + i + 1) if causal else length
            if lim <= 0:
                continue
            e = s[i, :, :lim]
            p = np.exp(e - e.max(-1, keepdims=True))
            out[i, h * G:(h + 1) * G] = p @ vv[:lim] / p.sum(-1, keepdims=True)
    return out


def decoded_heads(k: np.ndarray, v: np.ndarray, bits: int, group: int):
    """k, v [H, n, D] float32 -> the values their packed form stands for."""
    kd = np.stack([O.unpack_matrix(O.pack_k(x, bits, group)) for x in k])
    vd = np.stack([O.unpack_matrix(O.pack_v(x, bits, group)) for x in v])
    return kd, vd
