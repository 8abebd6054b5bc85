"""Plain numpy reference, in fp64, of the dense caches that stay bounded over a
session: attention of packed prompts, the weight that positions receive, and
eviction by it."""
from __future__ import annotations

import numpy as np

D = 128


def scores(q, k, scale, before):
    """Masked scores [Hq, n, L] of q [n, Hq, D] at positions before .. over
    k [Hkv, L, D]; and their largest sum of magnitudes, |scale| sum |q| |k|,
    over the positions each row sees, [Hq, n]."""
    n, Hq = q.shape[:2]
    R, L = Hq // k.shape[0], k.shape[1]
    late = np.arange(L) > before + np.arange(n)[:, None]
    a = np.empty((Hq, n, L))
    size = np.empty((Hq, n))
    for h in range(Hq):
        a[h] = np.where(late, -np.inf, scale * (q[:, h] @ k[h // R].T))
        size[h] = np.where(late, 0.0, abs(scale) * (np.abs(q[:, h]) @ np.abs(k[h // R]).T)).max(-1, initial=0.0)
    return a, size


def log_sum(a):
    """ln sum exp over the last axis."""
    top = a.max(-1, keepdims=True)
    return (top + np.log(np.exp(a - top).sum(-1, keepdims=True)))[..., 0]


def attend(q, k, v, scale, before):
    """(out [n, Hq, D], lse [n, Hq], sum_p softmax_p |v_p| [n, Hq, D], largest score magnitude [n, Hq])."""
    R = q.shape[1] // k.shape[0]
    a, size = scores(q, k, scale, before)
    lse = log_sum(a)
    out, mag = np.empty(q.shape), np.empty(q.shape)
    for h in range(q.shape[1]):
        w = np.exp(a[h] - lse[h][:, None])
        out[:, h], mag[:, h] = w @ v[h // R], w @ np.abs(v[h // R])
    return out, lse.T, mag, size.T


def received(q, k, scale, before, lse, window):
    """The weight that each position receives from the last `window` rows,
    [Hkv, L], given the rows' lse [n, Hq]."""
    n, Hq = q.shape[:2]
    Hkv = k.shape[0]
    first = max(0, n - window)
    if first == n:
        return np.zeros(k.shape[:2])
    a, _ = scores(q[first:], k, scale, before + first)
    return np.exp(a - lse[first:].T[..., None]).reshape(Hkv, Hq // Hkv, n - first, -1).sum((1, 2))


def kept(acc, keep, recent):
    """The positions of acc [L] that stay: the last `recent` and of the older
    ones the keep - recent largest (ties: the lowest; NaN: the largest)."""
    L = len(acc)
    if L <= keep:
        return list(range(L))
    old = sorted(range(L - recent), key=lambda p: (0 if np.isnan(acc[p]) else 1, 0.0 if np.isnan(acc[p]) else -acc[p], p))
    return sorted(old[:keep - recent]) + list(range(L - recent, L))
