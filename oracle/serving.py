"""Rotary positions and serving from a nested KV cache: the CPU oracle.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Plain numpy in fp64,
straight from the formulas, one row or one sequence at a time:

  rotary     (a, b) -> m (a cos w - b sin w, a sin w + b cos w), w = pos theta_i
  cache      a row is (hi - 8) s (draft) or (16 (hi - 8) + (lo - 8)) s / 16
  attention  query i of sequence b over the prefix and own tokens
             t <= len - L + i: softmax(q k / sqrt(128)) v, and its log-sum-exp
  weights    acc[t] += sum of exp(q k_t / sqrt(128) - lse) over the rows that see t
  eviction   first tokens, last tokens and the best of the rest, ties to the first
"""
from __future__ import annotations

import math

import numpy as np

D = 128


def rope_theta(rot, base, scaling="plain", factor=1.0, low=1.0, high=4.0, trained=0):
    """(theta fp64 [rot / 2], magnitude)."""
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2.0))
    theta = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == "linear":
        return theta / factor, 1.0
    if scaling == "bands":
        t = np.clip((trained * theta / (2 * math.pi) - low) / (high - low), 0.0, 1.0)
        return theta * (t + (1.0 - t) / factor), 1.0
    if scaling == "yarn":
        at = [rot * math.log(trained / (2 * math.pi * n)) / (2.0 * math.log(base))
              for n in (high, low)]
        first, last = max(0.0, math.floor(at[0])), min(rot - 1.0, math.ceil(at[1]))
        r = np.clip((np.arange(rot // 2) - first) / max(last - first, 1e-3), 0.0, 1.0)
        return theta * (1.0 - r + r / factor), 0.1 * math.log(factor) + 1.0
    return theta, 1.0


def angles(phases, pos):
    """fp64 angles [M, rot / 2] in (-pi, pi] from 64-bit phases, in Python's integers."""
    out = np.empty((len(pos), len(phases)))
    for m, p in enumerate(pos):
        for i, f in enumerate(phases):
            turn = (int(f) * int(p)) % (1 << 64)
            out[m, i] = 2 * math.pi * ((turn - (1 << 64) if turn >> 63 else turn) / 2.0 ** 64)
    return out


def rope(x, w, magnitude, layout, inverse=False):
    """x [M, heads, D] turned by angles w [M, rot / 2]; layout "half" or "pairs"."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    half = w.shape[1]
    c = magnitude * np.cos(w)[:, None]
    s = magnitude * np.sin(w)[:, None] * (-1.0 if inverse else 1.0)
    i = np.arange(half)
    a, b = (i, i + half) if layout == "half" else (2 * i, 2 * i + 1)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def values(mode, planes):
    """fp64 rows [..., 128] of (hi, lo, scale)."""
    hi, lo, sc = planes
    u = np.empty(hi.shape[:-1] + (D,))
    for k, shift in ((0, 0), (1, 4)):
        h = ((hi >> shift) & 15).astype(np.float64) - 8.0
        u[..., k::2] = h if mode == 0 else h + (((lo >> shift) & 15).astype(np.float64) - 8.0) / 16.0
    return u * sc.astype(np.float64)[..., None]


def attention(mode, q, prefix, own, lens):
    """(out, lse, size) fp64: size [B, L, H, 128] = sum p |v|, the scale of out's rounding."""
    B, L, H, _ = q.shape
    q = np.asarray(q, np.float64)
    out, size = np.zeros(q.shape), np.zeros(q.shape)
    lse = np.full((B, L, H), -np.inf)
    some = prefix or own
    Hkv = some[0][0].shape[-2]
    kp, vp = (values(mode, x) for x in prefix) if prefix else (np.zeros((0, Hkv, D)),) * 2
    for b in range(B):
        n = int(lens[b])
        if n < 0:
            continue
        if own:
            n = min(n, own[0][0].shape[1])
            ko, vo = (values(mode, tuple(a[b, :n] for a in x)) for x in own)
        for i in range(L):
            m = max(0, n - L + i + 1) if own else 0
            for h in range(H):
                j = h // (H // Hkv)
                k = np.concatenate([kp[:, j], ko[:m, j]]) if own else kp[:, j]
                v = np.concatenate([vp[:, j], vo[:m, j]]) if own else vp[:, j]
                if not len(k):
                    continue
                s = k @ q[b, i, h] / math.sqrt(D)
                top = s.max()
                p = np.exp(s - top)
                lse[b, i, h] = top + math.log(p.sum())
                p /= p.sum()
                out[b, i, h], size[b, i, h] = p @ v, p @ np.abs(v)
    return out, lse, size


def weights(mode, q, lse, k_planes, acc, lens=None):
    """acc [B, Hkv, cap] (lens None: [Hkv, P]) with the weights received added, fp64."""
    q, acc = np.asarray(q, np.float64), np.array(acc, np.float64)
    B, L, H, _ = q.shape
    k = values(mode, k_planes)
    Hkv = k.shape[-2]
    for b in range(B):
        for i in range(L):
            for h in range(H):
                j = h // (H // Hkv)
                if lse[b, i, h] == -np.inf:
                    continue
                kk = k[:, j] if lens is None else k[b, :max(0, min(int(lens[b]), k.shape[1]) - L + i + 1), j]
                w = np.exp(kk @ q[b, i, h] / math.sqrt(D) - float(lse[b, i, h]))
                if lens is None:
                    acc[j] += w
                else:
                    acc[b, j, :len(w)] += w
    return acc


def evict(acc, n, keep, sinks, recent):
    """The kept places of one sequence and KV head, in order."""
    if n <= keep:
        return list(range(n))
    held = list(range(sinks)) + list(range(n - recent, n))
    rest = sorted(range(sinks, n - recent),
                  key=lambda t: (-acc[t] if acc[t] == acc[t] else np.inf, acc[t] != acc[t], t))
    return sorted(held + rest[:keep - sinks - recent])
