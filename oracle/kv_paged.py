"""Plain numpy reference of the paged 8-bit key/value cache: what
mamba2_kv_append leaves in the pages, and mamba2_attn_paged's outputs in fp64.

A block of 16 positions of one kv head shares one fp32 scale,
m = max(max |block|, 2^-100), scale = m / 448 (in fp32), code =
e4m3(448 x / m) to nearest even, and the rotation in fp32 operations as the
library's header states them, so that codes and scales are compared bit for
bit (`rotate` in fp64 gives the exact values for a bound)."""
from __future__ import annotations

import numpy as np

D = 128
BLOCK = 16
TINY = np.float32(2.0 ** -100)

# the value of every code 0 .. 255 (0x7F and 0xFF are NaN)
_code = np.arange(256)
_e, _m = (_code >> 3) & 15, _code & 7
E4M3 = np.where(_e == 0, np.ldexp(_m / 8.0, -6), np.ldexp(1 + _m / 8.0, _e - 7)) * np.where(_code & 128, -1.0, 1.0)
E4M3[[0x7F, 0xFF]] = np.nan


def to_e4m3(x):
    """Codes of fp32 values to nearest even, saturating at 448."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    with np.errstate(invalid="ignore", divide="ignore"):
        e = np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -6.0)
    step = np.exp2(e - 3)
    q = np.rint(a / step) * step  # np.rint: ties to even
    e = np.where(q > 0, np.maximum(np.floor(np.log2(np.where(q > 0, q, 1.0))), -6.0), -6.0)
    m = np.nan_to_num(q / np.exp2(e))  # in [1, 2), or below 1 where subnormal
    code = np.where(m >= 1, (e + 7) * 8 + (m - 1) * 8, m * 8)
    code = np.nan_to_num(code).astype(np.int64) | np.where(np.signbit(x), 128, 0)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def _pairs(rot, interleaved):
    h = rot // 2
    i = np.arange(h)
    return (2 * i, 2 * i + 1) if interleaved else (i, h + i)


def rotate(x, places, cos, sin, rot, interleaved, dtype=np.float32):
    """x [..., n, heads, D] at positions `places` [n]; every product and sum
    rounded to dtype (fp32: the library's arithmetic)."""
    x = np.array(x, dtype)
    if not rot:
        return x
    a, b = _pairs(rot, interleaved)
    c, s = cos[places].astype(dtype)[:, None], sin[places].astype(dtype)[:, None]
    u, w = x[..., a].copy(), x[..., b].copy()
    x[..., a] = u * c - w * s
    x[..., b] = u * s + w * c
    return x


def quantise(rows):
    """rows [n, heads, D] fp32 from a block's first position on: codes of the
    same shape and scales [ceil(n / 16), heads]."""
    rows = np.asarray(rows, np.float32)
    n, H = rows.shape[:2]
    codes, scales = np.empty((n, H, D), np.uint8), np.empty((-(-n // BLOCK), H), np.float32)
    for i in range(scales.shape[0]):
        block = rows[i * BLOCK:(i + 1) * BLOCK]
        m = np.maximum(np.abs(block).max((0, 2)), TINY).astype(np.float32)
        scales[i] = m / np.float32(448)
        # 448 x is exact in fp64, and a quotient of fp32 numbers is no nearer than
        # 2^-50 of itself to a value halfway between two codes unless it is one
        codes[i * BLOCK:(i + 1) * BLOCK] = to_e4m3(block.astype(np.float64) * 448 / m.astype(np.float64)[:, None])
    return codes, scales


def read(pages, scales, table_row, page_size, n):
    """Positions 0 .. n - 1 of a session in fp64, [n, heads, D]."""
    p = np.arange(n)
    page, slot = np.asarray(table_row)[p // page_size], p % page_size
    with np.errstate(invalid="ignore"):
        return E4M3[pages[page, :, slot]] * scales[page, :, slot // BLOCK].astype(np.float64)[..., None]


def attend(q, k, v, scale, seen, vs=None):
    """fp64 outputs of q [n, Hq, D] over k, v [L, Hkv, D], query t over the
    first seen[t] positions; also what error bounds are made of, for each row:
    sum_p softmax_p |v_p|, the largest |scale| sum |q| |k|, and (with the
    values' scales vs [L, Hkv]) max_p(softmax_p vs_p) sum_p |v_p| / vs_p."""
    n, Hq = q.shape[:2]
    R = Hq // k.shape[1]
    out, size, reach, floor = np.zeros((n, Hq, D)), np.zeros((n, Hq, D)), np.zeros((n, Hq, 1)), np.zeros((n, Hq, D))
    for t in range(n):
        L = seen[t]
        if L == 0:
            continue
        for h in range(Hq):
            kk, vv = k[:L, h // R], v[:L, h // R]
            a = scale * (kk @ q[t, h])
            w = np.exp(a - a.max())
            w /= w.sum()
            out[t, h], size[t, h] = w @ vv, w @ np.abs(vv)
            reach[t, h] = abs(scale) * (np.abs(kk) @ np.abs(q[t, h])).max()
            if vs is not None:
                floor[t, h] = (w * vs[:L, h // R]).max() * (np.abs(vv) / vs[:L, h // R, None]).sum(0)
    return out, size, reach, floor
