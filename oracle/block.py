"""The operators around the routed experts written out from their definitions.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).  All arithmetic in
float64; a result that the definition rounds is given unrounded unless the
function says otherwise.
"""
from __future__ import annotations

import math
from typing import Optional, Tuple

import numpy as np

from . import codecs as C


def add_rmsnorm(x, gain: Optional[np.ndarray], eps: float, res=None) -> Tuple[np.ndarray, np.ndarray]:
    """(y, n): y = x + res, n = y / sqrt(mean(y^2) + eps) * gain, per row."""
    y = np.asarray(x, dtype=np.float64)
    if res is not None:
        y = y + np.asarray(res, dtype=np.float64)
    n = y / np.sqrt(np.mean(y * y, axis=-1, keepdims=True) + eps)
    return y, n if gain is None else n * np.asarray(gain, dtype=np.float64)


def scores(logits: np.ndarray, score: str) -> np.ndarray:
    """softmax over the row or sigmoid; 0 for a masked (-inf) or NaN logit."""
    l = np.asarray(logits, dtype=np.float64)
    out = np.zeros_like(l)
    for t in range(l.shape[0]):
        live = [e for e in range(l.shape[1]) if l[t, e] > -np.inf]  # false for NaN
        if not live:
            continue
        if score == "sigmoid":
            for e in live:
                out[t, e] = 1.0 / (1.0 + math.exp(-l[t, e])) if l[t, e] > -700 else 0.0
        else:
            top = max(l[t, e] for e in live)
            z = {e: 1.0 if l[t, e] == top else math.exp(l[t, e] - top) for e in live}
            total = sum(z.values())
            for e in live:
                out[t, e] = z[e] / total
    return out


def route_scored(logits, k: int, bias=None, score: str = "softmax", n_group: int = 1, topk_group: int = 1,
                 group_top: int = 1, renorm: bool = True, scale: float = 1.0):
    """(ids int32 [T,k], w float64 [T,k], any NaN).  Selection by c = s + bias;
    a -inf logit has c = -inf, a NaN logit or c ranks below that."""
    l = np.asarray(logits, dtype=np.float32)
    T, E = l.shape
    s = scores(l, score)
    per = E // n_group
    ids = np.zeros((T, k), dtype=np.int32)
    w = np.zeros((T, k))
    nan = False
    for t in range(T):
        c = [s[t, e] + (0.0 if bias is None else float(bias[e])) for e in range(E)]
        for e in range(E):
            if l[t, e] == -np.inf:
                c[e] = -np.inf
            if np.isnan(l[t, e]) or np.isnan(c[e]):
                c[e] = math.nan
                nan = True
        groups = list(range(n_group))
        if n_group > 1:
            best = []
            for g in range(n_group):
                v = sorted([-np.inf if np.isnan(v) else v for v in c[g * per:(g + 1) * per]], reverse=True)
                best.append(sum(v[:group_top]))
            groups = sorted(groups, key=lambda g: (-best[g], g))[:topk_group]
        cand = [e for e in range(E) if e // per in groups]
        cand.sort(key=lambda e: (np.isnan(c[e]), -c[e] if not np.isnan(c[e]) else 0.0, e))
        ids[t] = cand[:k]
        w[t] = s[t, ids[t]]
        if renorm:
            total = w[t].sum()
            w[t] = w[t] / total if total > 0 else 0.0
    return ids, w * scale, nan


def linear(x, w, bias=None, act: str = "none", res=None) -> np.ndarray:
    """act(x w^T + bias) + res; swiglu: w = gate rows, then up rows."""
    v = np.asarray(x, dtype=np.float64) @ np.asarray(w, dtype=np.float64).T
    if bias is not None:
        v = v + np.asarray(bias, dtype=np.float64)
    sig = lambda a: 0.5 * (1.0 + np.tanh(0.5 * a))  # noqa: E731
    if act == "silu":
        v = v * sig(v)
    elif act == "gelu":
        v = 0.5 * v * (1.0 + np.vectorize(math.erf)(v / math.sqrt(2.0)))
    elif act == "swiglu":
        n = v.shape[1] // 2
        v = v[:, :n] * sig(v[:, :n]) * v[:, n:]
    return v if res is None else v + np.asarray(res, dtype=np.float64)


def mxfp8_rows(out_bf16_bits: np.ndarray):
    """MXFP8 codes and scales of bf16 rows (bit patterns)."""
    return C.mxfp8_quantize(C.bf16_bits_to_f64(out_bf16_bits))
