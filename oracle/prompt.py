"""The operators of a layer over packed prompts, in float64 (TEST INFRASTRUCTURE,
oracle): causal attention with grouped heads, rotary positions with several
axes, and the linear layers with an epilogue.

Only the test suite may import this module.  Pinned by
``tests/test_oracle_prompt.py``.
"""
from __future__ import annotations

import math
from typing import Optional, Sequence

import numpy as np

from .attention import to_f64


def prompt_attention(q, k, v, lengths_q: Sequence[int], lengths_k: Sequence[int], causal: bool,
                     scale: float, rows: Optional[Sequence[int]] = None):
    """q [Tq, Hq, D], k and v [Tk, Hkv, D].  Query i of a sequence sees key j iff
    j <= Lk - Lq + i (causal) or every key; query head h reads K/V head
    h // (Hq // Hkv); a query that sees no key gives zeros.  Returns (out,
    weight, reach) for the packed rows `rows` (all): weight = sum_j w_j |v_j|
    (what relative errors of the weights multiply) and reach = max_j |scale|
    sum_d |q_d k_jd| (what relative errors of the scores multiply)."""
    q, k, v = to_f64(q), to_f64(k), to_f64(v)
    Hq, D = q.shape[1:]
    G = Hq // k.shape[1]
    rows = np.arange(sum(lengths_q)) if rows is None else np.asarray(rows, dtype=np.int64)
    out = np.zeros((len(rows), Hq, D))
    weight, reach = np.zeros_like(out), np.zeros((len(rows), Hq, 1))
    q0 = k0 = 0
    for lq, lk in zip(lengths_q, lengths_k):
        mine = np.nonzero((rows >= q0) & (rows < q0 + lq))[0]
        if len(mine) and lk:
            i = rows[mine] - q0
            seen = np.arange(lk)[None, :] <= (lk - lq + i)[:, None] if causal else \
                np.ones((len(i), lk), dtype=bool)
            for h in range(Hq):
                x, kh, vh = q[rows[mine], h], k[k0:k0 + lk, h // G], v[k0:k0 + lk, h // G]
                s = np.where(seen, (x @ kh.T) * scale, -np.inf)
                top = s.max(axis=1, keepdims=True)
                w = np.where(seen, np.exp(s - np.where(np.isfinite(top), top, 0.0)), 0.0)
                den = w.sum(axis=1, keepdims=True)
                w = np.where(den > 0, w / np.where(den > 0, den, 1.0), 0.0)
                out[mine, h] = w @ vh
                weight[mine, h] = w @ np.abs(vh)
                size = np.where(seen, (np.abs(x) @ np.abs(kh).T) * abs(scale), 0.0)
                reach[mine, h, 0] = size.max(axis=1)
        q0, k0 = q0 + lq, k0 + lk
    return out, weight, reach


def axis_angles(positions, axis_dims: Sequence[int], base: float, shared: bool) -> np.ndarray:
    """Angles [T, R/2] of every token's pairs; positions [axes, T], R = sum(axis_dims)."""
    pos = np.asarray(positions, dtype=np.float64)
    R, cols, first = sum(axis_dims), [], 0
    for a, d in enumerate(axis_dims):
        for j in range(d // 2):
            power = 2.0 * (first + j) / R if shared else 2.0 * j / d
            cols.append(pos[a] * float(base) ** -power)
        first += d // 2
    return np.stack(cols, axis=1)


def rope_axes(x, positions, axis_dims: Sequence[int], base: float, halves: bool = False,
              shared: bool = False) -> np.ndarray:
    """x [T, H, D] with the first R elements of every head turned pair by pair."""
    x = to_f64(x)
    z = axis_angles(positions, axis_dims, base, shared)
    c, s = np.cos(z)[:, None, :], np.sin(z)[:, None, :]
    R = 2 * z.shape[1]
    first = np.arange(R // 2) if halves else np.arange(0, R, 2)
    second = first + (R // 2 if halves else 1)
    out = x.copy()
    out[..., first] = x[..., first] * c - x[..., second] * s
    out[..., second] = x[..., first] * s + x[..., second] * c
    return out


_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def activation(v: np.ndarray, name: str) -> np.ndarray:
    v = np.asarray(v, dtype=np.float64)
    if name == "relu":
        return np.maximum(v, 0.0)
    if name == "silu":
        return v * _logistic(v)
    if name == "gelu":
        return 0.5 * v * _erfc(-v / math.sqrt(2.0))
    if name == "gelu_tanh":
        # (1 + tanh u) / 2 is the logistic function of 2 u
        return v * _logistic(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))
    if name != "none":
        raise ValueError(name)
    return v


def _logistic(t: np.ndarray) -> np.ndarray:
    e = np.exp(-np.abs(t))
    return np.where(t >= 0, 1.0, e) / (1.0 + e)


def linear_act(x, w, bias=None, act: str = "none", residual=None):
    """(residual + act(x w^T + bias), size): size = sum_k |x_k w_k| + |bias|,
    what relative errors of the product's sums multiply."""
    x, w = to_f64(x), to_f64(w)
    v, size = x @ w.T, np.abs(x) @ np.abs(w).T
    if bias is not None:
        v, size = v + to_f64(bias), size + np.abs(to_f64(bias))
    y = activation(v, act)
    return (y if residual is None else y + to_f64(residual)), size


def linear_gated(x, w_gate, w_up, act: str = "silu"):
    """act(x w_gate^T) * (x w_up^T), and the two factors with their sizes:
    (y, gate, size of the gate's sums, up, size of up's sums)."""
    gate, gate_size = linear_act(x, w_gate)
    up, up_size = linear_act(x, w_up)
    return activation(gate, act) * up, gate, gate_size, up, up_size
