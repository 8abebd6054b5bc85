"""The forms of mamba2_attn_paged, each in cases that are checked to take it: the
tiles alone and shared by two, four and eight CTAs, the rows form alone and
shared, runs of positions longer than the page numbers that are read at once,
and page tables much wider than their sessions.

References in fp64 on the GPU, from what the cache holds; the tolerances are
those that stand at the head of test_gpu_kv_paged.py, with queries that may be
off by 2^-21 of a row's largest."""
import ctypes

import numpy as np
import pytest

from test_gpu_kv_paged import BLOCK, D, Cache, _int, _rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m2():
    import full_duplex_speech_gb300 as m2
    m2.load()
    return m2


def plan(m2, cache, T, Hq):
    """(form, CTAs that share a set of rows' positions) of a call."""
    code = m2.load().m2_attn_paged_plan(ctypes.byref(cache.desc), T, Hq)
    assert code > 0, code
    return ("tiles" if code >= 256 else "rows"), code % 256


def cached(cache, s, n):
    """Keys, values and the values' scales of session s in fp64 on the GPU."""
    import torch
    p = torch.arange(n, device="cuda")
    page, slot = cache.d_table[s].long()[p // cache.ps], p % cache.ps

    def read(codes, scales):
        c = codes.view(torch.float8_e4m3fn)[page, :, slot].double()
        sc = scales[page, :, slot // BLOCK].double()
        return c * sc[..., None], sc

    k, v = read(cache.kp, cache.ks), read(cache.vp, cache.vs)
    return k[0], v[0], v[1]


def attend64(q, k, v, scale, seen):
    """q [n, Hq, D], k, v [L, Hkv, D] in fp64; query t over the first seen[t]
    positions. Outputs, the softmax and |scale| sum |q| |k| at its largest."""
    import torch
    n, Hq = q.shape[:2]
    R = Hq // k.shape[1]
    hidden = torch.arange(k.shape[0], device="cuda") >= torch.as_tensor(seen, device="cuda")[:, None]
    out, weights, reach = [], [], []
    for h in range(Hq):
        a = (scale * (q[:, h] @ k[:, h // R].T)).masked_fill(hidden, -np.inf)
        w = torch.nan_to_num(torch.softmax(a, -1))
        reach.append(abs(scale) * (q[:, h].abs() @ k[:, h // R].abs().T).masked_fill(hidden, 0).amax(-1))
        out.append(w @ v[:, h // R])
        weights.append(w)
    return torch.stack(out, 1), weights, torch.stack(reach, 1)[..., None]


def check(cache, q, got, lengths, new, causal, scale, act):
    import torch
    for s, (L, n) in enumerate(zip(lengths, new)):
        assert bool((got[s, n:] == -7.0).all()), "rows behind the last are left as they were"
        if n == 0:
            continue
        if not causal and L == 0:
            assert not bool(got[s, :n].any()), "rows that see nothing are zeros"
            continue
        k, v, vs = cached(cache, s, L + n if causal else L)
        qd = q[s, :n].double()
        seen = [L + t + 1 if causal else L for t in range(n)]
        want, weights, A = attend64(qd, k, v, scale, seen)
        R = q.shape[2] // k.shape[1]
        S = torch.stack([w @ v[:, h // R].abs() for h, w in enumerate(weights)], 1)
        W = torch.stack([(w * vs[:, h // R]).amax(-1, keepdim=True) * (v[:, h // R].abs() / vs[:, h // R, None]).sum(0)
                         for h, w in enumerate(weights)], 1)
        d = 128 * 2.0 ** -24 * A
        if act == "bf16":
            wide = k.abs().sum(-1).amax(0).repeat_interleave(R)[:, None]
            d = d + 2.0 ** -21 * qd.abs().amax(-1, keepdim=True) * abs(scale) * wide
            tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 1e-5 + 2 * d) * S
        else:
            tol = 2.0 ** -24 * want.abs() + (2.0 ** -21 + 1e-5 + 2 * (d + 2.0 ** -21 * A)) * S
        tol = tol + 2.0 ** (-25 if act == "bf16" else -40) * W + 2.0 ** -126 * (1 + v.abs().sum(0).repeat_interleave(R, 0))
        err = (got[s, :n].double() - want).abs()
        assert bool(torch.isfinite(got[s, :n]).all())
        assert bool((err <= tol).all()), (s, float((err - tol).max()))


def fill(m2, seed, S, Hkv, ps, act, reach, capacity):
    cache = Cache(m2, S, Hkv, ps, capacity, act, seed=seed)
    T = max(max(reach), 1)
    (k, _), (v, _) = _rows(seed + 1, S, T, Hkv, act), _rows(seed + 2, S, T, Hkv, act)
    cache.append(k, v, _int(reach))
    return cache


@pytest.mark.parametrize("form,W,act,ps,Hq,Hkv,lengths,T,capacity", [
    # tiles, runs of more than 32 page numbers (pages of 16: 8 a chunk of 128 positions)
    ("tiles", 1, "bf16", 16, 64, 32, [1100], 512, 0),
    ("tiles", 2, "bf16", 16, 80, 16, [1900], 200, 0),
    ("tiles", 4, "bf16", 16, 40, 8, [3300], 200, 0),
    ("tiles", 8, "bf16", 16, 10, 2, [5200], 200, 0),
    ("tiles", 1, "bf16", 128, 76, 38, [4700], 512, 0),
    ("tiles", 8, "bf16", 128, 10, 2, [5200], 200, 0),
    ("tiles", 1, "bf16", 16, 80, 16, [700, 0, 1301, 64, 900], 300, 0),
    # the rows form, alone and shared, a few rows and sixteen at a time
    ("rows", 1, "bf16", 16, 160, 32, [900, 0, 31, 1500] * 4, 1, 0),
    ("rows", 16, "bf16", 16, 5, 1, [9000], 1, 0),
    ("rows", 16, "bf16", 16, 5, 1, [9000], 7, 0),
    ("rows", 16, "f32", 128, 5, 1, [9000], 4, 0),
    # page tables for 8,000 positions and more, and sessions of a few
    ("rows", 16, "bf16", 64, 5, 1, [300, 0], 1, 8000),
    ("rows", 16, "f32", 16, 5, 1, [300], 3, 8000),
    ("tiles", 8, "bf16", 16, 10, 2, [300], 75, 8000),
    ("tiles", 8, "bf16", 64, 10, 2, [0, 300], 75, 60000),
    ("tiles", 8, "bf16", 32, 10, 2, [5], 100, 1 << 20),
])
def test_each_form(m2, form, W, act, ps, Hq, Hkv, lengths, T, capacity):
    S = len(lengths)
    rng = np.random.default_rng(T)
    new = [T] + [int(x) for x in rng.integers(0, T + 1, S - 1)]
    reach = [L + n for L, n in zip(lengths, new)]
    cache = fill(m2, 300 + T, S, Hkv, ps, act, reach, max(capacity, max(reach)))
    assert plan(m2, cache, T, Hq) == (form, W)
    q, _ = _rows(301 + T, S, T, Hq, act)
    for causal in (True, False):
        got = cache.attend(q, causal, _int(new), lengths=_int(lengths))
        check(cache, q, got, lengths, new, causal, D ** -0.5, act)
    assert m2.mamba2_device_error() == 0
