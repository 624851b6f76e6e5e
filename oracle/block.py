"""The block operators: expert choice with scores, bias and groups, the norms
around a block's end, dense products with their epilogues.

TEST INFRASTRUCTURE ONLY (see the package docstring). Everything is float64,
by plain loops over tokens where the definition is one of a choice.
"""
from __future__ import annotations

import math

import numpy as np

from .bf16 import bf16_rne

INF = float("inf")
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def sigmoid(v):
    v = np.asarray(v, dtype=np.float64)
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def scores(logits, score="softmax"):
    """Scores [T, E] of logits float64 [T, E]; 0 where a logit is NaN or -inf."""
    z = np.where(np.isnan(logits), -INF, np.asarray(logits, dtype=np.float64))
    if score == "sigmoid":
        return sigmoid(z)
    out = np.zeros_like(z)
    for t, row in enumerate(z):
        top = row.max()
        if top == INF:
            e = (row == INF).astype(np.float64)
        elif top == -INF:
            continue
        else:
            e = np.exp(row - top)
        out[t] = e / math.fsum(e)
    return out


def route_experts(logits, k, score="softmax", bias=None, groups=1, top_groups=None,
                  group_score="max", renormalize=True, scale=1.0):
    """(ids int32 [T, k], w float64 [T, k])."""
    z = np.where(np.isnan(logits), -INF, np.asarray(logits, dtype=np.float64))
    T, E = z.shape
    s = scores(z, score)
    ids, w = np.full((T, k), -1, dtype=np.int32), np.zeros((T, k))
    top_groups = groups if top_groups is None else top_groups
    per = E // groups
    for t in range(T):
        # experts in the order of choice: key descending, index ascending
        key = {}
        for e in range(E):
            v = z[t, e] if bias is None else s[t, e] + float(bias[e])
            if z[t, e] > -INF and v > -INF:
                key[e] = v
        if groups > 1 and top_groups < groups:
            # without a bias groups of one score each compare by logits too
            ranked = []
            for g in range(groups):
                mine = sorted((key[e] if bias is not None or group_score == "max" else s[t, e]
                               for e in range(g * per, (g + 1) * per) if e in key), reverse=True)
                if mine:
                    ranked.append((-sum(mine[:2]) if group_score == "top2" else -mine[0], g))
            kept = {g for _, g in sorted(ranked)[:top_groups]}
            key = {e: v for e, v in key.items() if e // per in kept}
        chosen = sorted(key, key=lambda e: (-key[e], e))[:k]
        ids[t, :len(chosen)] = chosen
        v = s[t, chosen]
        if renormalize:
            total = v.sum()
            v = v / total if total > 0 else v
        w[t, :len(chosen)] = scale * v
    return ids, w


def norm(v, weight, eps, offset=0.0):
    v = np.asarray(v, dtype=np.float64)
    return v / np.sqrt(np.mean(v * v, axis=-1, keepdims=True) + eps) * (weight + offset)


def norm_add(x, residual, post=None, gate=None, gate_fn=None, scale=1.0, residual_scale=1.0,
             eps=1e-6, unit_offset=False):
    """(t, p): the residual stream before its rounding to bf16, and the gated
    and scaled branch in it. gate broadcasts against [T, H]."""
    off = 1.0 if unit_offset else 0.0
    p = np.asarray(x, dtype=np.float64) if post is None else norm(x, post, eps, off)
    if gate is not None:
        p = p * {None: lambda g: g, "sigmoid": sigmoid, "tanh": np.tanh}[gate_fn](
            np.asarray(gate, dtype=np.float64))
    p = scale * p
    return residual_scale * residual + p, p


def activate(y, activation=None):
    if activation is None:
        return y
    if activation == "relu":
        return np.maximum(y, 0.0)
    if activation == "silu":
        return y * sigmoid(y)
    if activation == "gelu":
        return 0.5 * y * _erfc(-y / math.sqrt(2))   # (1 + erf z = erfc -z)
    if activation == "gelu_tanh":
        return y * sigmoid(math.sqrt(8 / math.pi) * (y + 0.044715 * y ** 3))   # (1 + tanh z) / 2
    I = y.shape[1] // 2
    return y[:, :I] * sigmoid(y[:, :I]) * y[:, I:]


def dense(x, weight, bias=None, activation=None, residual=None):
    """(out, Y, S) before rounding: the result, the product with its bias, and the
    sum of magnitudes, which bounds what an FP32 sum can lose."""
    S = np.abs(x) @ np.abs(weight).T
    Y = x @ weight.T
    if bias is not None:
        Y, S = Y + bias, S + np.abs(bias)
    out = activate(Y, activation)
    return (out if residual is None else out + residual), Y, S


__all__ = ["sigmoid", "scores", "route_experts", "norm", "norm_add", "activate", "dense", "bf16_rne"]
