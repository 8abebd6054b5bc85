"""GPU parity of the paged 8-bit cache (mamba2_kv_append, mamba2_attn_paged)
against its plain reference (oracle/kv_paged.py), through the C ABI.

Tolerances.
  Append: codes, scales and tails are compared bit for bit with the fp32
    formula of the header (rotated queries too, rounded once to bf16).
  Attention, per element, with S = sum_p softmax_p |v_p| and A the row's
    largest |scale| sum |q| |k|:
      scores  an fp32 sum of 128 products in any order is off by at most
              128 x 2^-24 A; bf16 queries may enter the product as two e4m3
              terms, off by at most 2^-17 max|q| a dim, so by
              2^-17 max|q| |scale| sum |k|; fp32 queries as two fp16 terms,
              2^-21 A. With d the sum of these, a softmax weight moves by
              2 d of itself, so the output by 2 d S.
      weights rounded to fp16 for bf16 activations, 2^-11 S; as two fp16
              terms for fp32, 2^-21 S; plus exp2 and the fp32 sums, 1e-5 S
              (positions in the hundreds, 2^-24 each, and 2^-22 for exp2).
              fp16 weights enter relative to at least 1 (fp32: 2^15) over
              the largest product W of a weight and its value's scale and
              are subnormal below 2^-14, so each is off by at most 2^-25:
              2^-25 W sum |code| (fp32: 2^-40).
              A weight below 2^-126 of the largest is zero in fp32:
              2^-126 sum |v|, and 2^-126 for outputs below the normals.
      output  rounded once: 2^-8 |out| in bf16, 2^-24 in fp32."""
import math

import numpy as np
import pytest

from oracle import kv_paged as kv

pytestmark = pytest.mark.gpu

D, BLOCK = kv.D, kv.BLOCK


@pytest.fixture(scope="module")
def m2():
    import full_duplex_speech_gb300 as m2
    m2.load()
    return m2


def _dt(act):
    import torch
    return torch.bfloat16 if act == "bf16" else torch.float32


class Cache:
    """A pool on the GPU with NaN codes and scales wherever nothing was written."""

    def __init__(self, m2, S, Hkv, ps, capacity, act, seed=0, spare=3, in_place=True):
        import torch
        self.m2, self.S, self.Hkv, self.ps, self.act = m2, S, Hkv, ps, act
        self.columns = max(1, -(-capacity // ps))
        self.n_pages = S * self.columns + spare
        rng = np.random.default_rng(seed)
        self.table = rng.permutation(self.n_pages)[:S * self.columns].reshape(S, self.columns).astype(np.int32)
        dev = dict(device="cuda")
        self.d_table = torch.from_numpy(self.table).cuda()
        self.kp, self.vp = (torch.full((self.n_pages, Hkv, ps, D), 0x7F, dtype=torch.uint8, **dev) for _ in "kv")
        self.ks, self.vs = (torch.full((self.n_pages, Hkv, ps // BLOCK), math.nan, **dev) for _ in "kv")
        self.kt, self.vt = (torch.full((S, Hkv, BLOCK, D), math.nan, **dev) for _ in "kv")
        self.kto, self.vto = (self.kt, self.vt) if in_place else (t.clone() for t in (self.kt, self.vt))
        self.lengths = torch.zeros(S, dtype=torch.int32, **dev)
        self.desc = m2.kv_cache(S, Hkv, ps, self.n_pages, self.columns, self.d_table, self.kp, self.vp, self.ks, self.vs,
                                self.kt, self.vt, self.kto, self.vto, act=act)

    def append(self, k, v, n_new=None, rope=None, q=None, lengths=None, stream=None, pad=0):
        """k, v [S, T, Hkv, D] (q [S, T, Hq, D]) as columns of q | k | v rows
        `pad` elements wider; returns the rotated q, -7 where not written."""
        import torch
        S, T = k.shape[:2]
        Hq = 0 if q is None else q.shape[2]
        width = (Hq + 2 * self.Hkv) * D + pad
        rows = torch.zeros(S, T, width, dtype=_dt(self.act), device="cuda")
        rows[..., :Hq * D] = 0 if q is None else q.reshape(S, T, -1)
        rows[..., Hq * D:(Hq + self.Hkv) * D] = k.reshape(S, T, -1)
        rows[..., (Hq + self.Hkv) * D:(Hq + 2 * self.Hkv) * D] = v.reshape(S, T, -1)
        out = None if q is None else torch.full((S, T, Hq * D + pad), -7.0, dtype=_dt(self.act), device="cuda")
        self.m2.mamba2_kv_append(self.desc, T, self.lengths if lengths is None else lengths, n_new, rows[0, 0, Hq * D:],
                                 rows[0, 0, (Hq + self.Hkv) * D:], width, rope, Hq, rows if Hq else None, width if Hq else 0,
                                 out, Hq * D + pad if Hq else 0, stream=stream)
        self._keep = rows
        return None if q is None else out[..., :Hq * D].view(S, T, Hq, D)

    def attend(self, q, causal=True, n_new=None, scale=None, lengths=None, pad=0, stream=None, out=None):
        import torch
        S, T, Hq = q.shape[:3]
        width = Hq * D + pad
        rows = torch.zeros(S, T, width, dtype=_dt(self.act), device="cuda")
        rows[..., :Hq * D] = q.reshape(S, T, -1)
        if out is None:
            out = torch.full((S, T, width), -7.0, dtype=_dt(self.act), device="cuda")
        ws = torch.empty(max(1, self.m2.mamba2_attn_paged_workspace_bytes(self.desc, T, Hq)), dtype=torch.uint8, device="cuda")
        self.m2.mamba2_attn_paged(self.desc, T, Hq, causal, self.lengths if lengths is None else lengths, n_new, rows, width,
                                  D ** -0.5 if scale is None else scale, out, width, ws, stream=stream)
        self._keep = (rows, ws)
        return out[..., :Hq * D].view(S, T, Hq, D)

    def host(self):
        return [t.cpu().numpy() for t in (self.kp, self.vp, self.ks, self.vs)]

    def read(self, s, n):
        kp, vp, ks, vs = self.host()
        return kv.read(kp, ks, self.table[s], self.ps, n), kv.read(vp, vs, self.table[s], self.ps, n)


def _int(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _rows(seed, S, T, H, act):
    """Keys, values or queries of uneven size, on the GPU and in fp32 numpy."""
    import torch
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(S, T, H, D)) * np.exp(rng.normal(size=(S, T, H, 1)) * 0.5) * np.exp(rng.normal(size=D) * 0.4)
    t = torch.from_numpy(x.astype(np.float32)).to(_dt(act))
    return t.cuda(), t.float().numpy()


def _rope(m2, rot, n_pos, interleaved):
    import torch
    if not rot:
        return None, None, None
    ang = np.arange(n_pos)[:, None] * 10000.0 ** -(np.arange(rot // 2) / (rot // 2))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    return m2.rope(rot, n_pos, torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda(), interleaved), cos, sin


def _expected_pool(cache, history):
    """Pool contents after `history` [s] = (k, v) fp32 [n, Hkv, D] rotated rows."""
    kp = np.full((cache.n_pages, cache.Hkv, cache.ps, D), 0x7F, np.uint8)
    vp, ks = kp.copy(), np.full((cache.n_pages, cache.Hkv, cache.ps // BLOCK), np.nan, np.float32)
    vs = ks.copy()
    for s, (k, v) in enumerate(history):
        for rows, pages, scales in ((k, kp, ks), (v, vp, vs)):
            codes, sc = kv.quantise(rows)
            p = np.arange(len(rows))
            pages[cache.table[s, p // cache.ps], :, p % cache.ps] = codes
            b = np.arange(0, len(rows), BLOCK)
            scales[cache.table[s, b // cache.ps], :, b % cache.ps // BLOCK] = sc
    return kp, vp, ks, vs


def _same(a, b):
    np.testing.assert_array_equal(np.ascontiguousarray(a).view(np.uint8), np.ascontiguousarray(b).view(np.uint8))


@pytest.mark.parametrize("act,ps,rot,interleaved,Hq,Hkv,steps,in_place,pad", [
    ("bf16", 64, 128, False, 40, 8, [[1, 1, 1], [16, 15, 14], [1, 1, 1], [1, 2, 0]], True, 0),
    ("bf16", 16, 0, False, 0, 1, [[3, 17, 0], [20, 0, 33], [70, 31, 64]], True, 8),
    ("f32", 32, 64, True, 4, 2, [[5, 40, 16], [43, 9, 0], [1, 1, 32]], True, 4),
    ("f32", 128, 16, False, 3, 1, [[130, 127, 128], [1, 1, 1]], False, 0),
    ("bf16", 128, 32, True, 6, 3, [[0, 0, 0], [2, 1, 150], [14, 15, 107]], False, 8),
])
def test_append_leaves_the_formulas_bits(m2, act, ps, rot, interleaved, Hq, Hkv, steps, in_place, pad):
    import torch
    S = len(steps[0])
    total = np.sum(steps, 0)
    cache = Cache(m2, S, Hkv, ps, int(total.max()), act, seed=5, in_place=in_place)
    rope, cos, sin = _rope(m2, rot, int(total.max()), interleaved)
    history = [(np.zeros((0, Hkv, D), np.float32),) * 2 for _ in range(S)]
    before = np.zeros(S, int)
    for i, new in enumerate(steps):
        T = max(1, max(new) + i % 2)  # padded rows behind the longest session too
        (k, kh), (v, vh) = _rows(10 + i, S, T, Hkv, act), _rows(30 + i, S, T, Hkv, act)
        q, qh = _rows(50 + i, S, T, Hq, act) if Hq else (None, None)
        got = cache.append(k, v, _int(new), rope, q, _int(before), pad=pad)
        for s, n in enumerate(new):
            places = before[s] + np.arange(n)
            kr = kv.rotate(kh[s, :n], places, cos, sin, rot, interleaved)
            history[s] = (np.concatenate((history[s][0], kr)), np.concatenate((history[s][1], vh[s, :n])))
            if Hq:
                want = torch.full((T, Hq, D), -7.0, dtype=_dt(act))
                want[:n] = torch.from_numpy(kv.rotate(qh[s, :n], places, cos, sin, rot, interleaved)).to(_dt(act))
                assert torch.equal(got[s].cpu(), want)
            left = (before[s] + n) % BLOCK
            for tail, rows in zip((cache.kto, cache.vto), history[s]):
                _same(tail[s, :, :left].cpu().numpy(), rows[len(rows) - left:].transpose(1, 0, 2))
        before += np.array(new)
        for a, b in zip(cache.host(), _expected_pool(cache, history)):
            _same(a, b)
        if not in_place:  # the next call reads what this one wrote
            cache.kt.copy_(cache.kto), cache.vt.copy_(cache.vto)
    assert m2.mamba2_device_error() == 0


def test_append_against_64_bits_and_extreme_blocks(m2):
    """Values within half an e4m3 step of the fp64 rotation (2^-4 of the value,
    2^-10 of the scale where subnormal, and 3 fp32 roundings of the rotation,
    of the products' size); blocks of zeros, of tiny and of huge values; an
    infinity or a NaN stays in its block."""
    import torch
    S, Hkv, T, ps = 1, 2, 96, 32
    cache = Cache(m2, S, Hkv, ps, T, "f32")
    rope, cos, sin = _rope(m2, 128, T, False)
    k, kh = _rows(3, S, T, Hkv, "f32")
    v, vh = _rows(4, S, T, Hkv, "f32")
    for t in (v, vh):
        t[0, 0:16, 0] = 0
        t[0, 16:32, 0] *= 1e-37
        t[0, 32:48, 0] *= 1e30
        t[0, 50, 0, 7] = math.inf
        t[0, 65, 1, 9] = math.nan
    cache.append(k, v, None, rope)
    kd, vd = cache.read(0, T)
    exact = kv.rotate(kh[0], np.arange(T), cos, sin, 128, False, np.float64)
    size = np.abs(kh[0]) + np.abs(np.roll(kh[0], 64, -1))
    _, _, ks, vs = cache.host()
    sk = ks[cache.table[0, np.arange(T) // ps], :, np.arange(T) % ps // BLOCK][..., None].astype(np.float64)
    sv = vs[cache.table[0, np.arange(T) // ps], :, np.arange(T) % ps // BLOCK][..., None].astype(np.float64)
    slack = 2.0 ** -4 + 2.0 ** -21
    assert np.all(np.abs(kd - exact) <= slack * np.abs(exact) + 2.0 ** -10 * sk + 3 * 2.0 ** -24 * size)
    whole = np.isfinite(sv) & np.isfinite(vh[0])
    with np.errstate(invalid="ignore"):
        near = np.abs(vd - vh[0]) <= slack * np.abs(vh[0]) + 2.0 ** -10 * sv
    bad = np.zeros((T, Hkv), bool)
    bad[48:64, 0] = bad[64:80, 1] = True
    assert np.all(near[~bad]) and np.all(whole[~bad])
    assert not np.isfinite(sv[bad]).any()
    assert np.all(vd[0:16, 0] == 0)


@pytest.mark.parametrize("power", [-95, 0, 70, 110])
def test_quotients_halfway_between_two_codes(m2, power):
    """448 x / m exactly halfway between two codes where 448 / m is not an fp32
    number (m = 21 x 2^power), and its fp32 neighbours on either side; codes
    subnormal and normal, blocks small and huge."""
    import torch
    mids = (kv.E4M3[:126] + kv.E4M3[1:127]) / 2
    x = (mids * 3 / 64).astype(np.float32)
    assert np.all(x.astype(np.float64) * 448 / 21 == mids)
    x = np.concatenate((x, np.nextafter(x, np.float32(0)), np.nextafter(x, np.float32(30))))
    rows = np.zeros((16, 1, D), np.float32)
    rows.reshape(-1)[:2 * len(x)] = np.concatenate((x, -x))
    rows[15, 0, 127] = 21
    rows = np.ldexp(rows, power)
    cache = Cache(m2, 1, 1, 16, 16, "f32")
    t = torch.from_numpy(rows[None]).cuda()
    cache.append(t, t)
    codes, scales = kv.quantise(rows)
    kp, vp, ks, vs = cache.host()
    page = cache.table[0, 0]
    for p, sc in ((kp, ks), (vp, vs)):
        _same(p[page, 0], codes[:, 0])
        _same(sc[page, 0], scales[0])


def test_cache_does_not_depend_on_the_split(m2):
    """One call, single frames, and odd pieces leave the same pool and tails."""
    S, Hkv, T, ps = 2, 2, 83, 16
    (k, _), (v, _) = _rows(1, S, T, Hkv, "bf16"), _rows(2, S, T, Hkv, "bf16")
    rope = _rope(m2, 128, T, False)[0]
    left = []
    for pieces in ([T], [1] * T, [7, 16, 9, 32, 1, 18]):
        cache = Cache(m2, S, Hkv, ps, T, "bf16")
        at = 0
        for n in pieces:
            cache.append(k[:, at:at + n], v[:, at:at + n], None, rope)
            cache.lengths += n
            at += n
        left.append(cache.host() + [cache.kt[:, :, :T % BLOCK].cpu().numpy(), cache.vt[:, :, :T % BLOCK].cpu().numpy()])
    for other in left[1:]:
        for a, b in zip(left[0], other):
            _same(a, b)


def test_queries_rotated_in_place(m2):
    import torch
    cache = Cache(m2, 2, 1, 16, 40, "bf16")
    rope, cos, sin = _rope(m2, 128, 40, False)
    q, qh = _rows(8, 2, 5, 3, "bf16")
    k = torch.zeros(2, 5, 1, D, dtype=torch.bfloat16, device="cuda")
    m2.mamba2_kv_append(cache.desc, 5, _int([3, 20]), _int([5, 4]), k, k, D, rope, 3, q, 3 * D, q, 3 * D)
    for s, (L, n) in enumerate([(3, 5), (20, 4)]):
        want = torch.from_numpy(qh[s]).clone()
        want[:n] = torch.from_numpy(kv.rotate(qh[s, :n], L + np.arange(n), cos, sin, 128, False))
        assert torch.equal(q[s].cpu(), want.to(torch.bfloat16))


# ------------------------------------------------------------------ attention

def _fill(m2, seed, S, Hkv, ps, act, reach, capacity=None):
    """A cache with reach[s] positions appended, everything else NaN."""
    cache = Cache(m2, S, Hkv, ps, max(capacity or 0, max(reach), 1), act, seed=seed)
    T = max(reach)
    if T:
        (k, _), (v, _) = _rows(seed + 1, S, T, Hkv, act), _rows(seed + 2, S, T, Hkv, act)
        cache.append(k, v, _int(reach))
    return cache


def _check(cache, q, got, lengths, new, causal, scale, act):
    got = got.float().cpu().numpy().astype(np.float64)
    qh = q.float().cpu().numpy().astype(np.float64)
    for s, (L, n) in enumerate(zip(lengths, new)):
        assert np.all(got[s, n:] == -7.0), "rows behind the last are left as they were"
        if n == 0:
            continue
        k, v = cache.read(s, L + n if causal else L)
        seen = [L + t + 1 if causal else L for t in range(n)]
        p = np.arange(len(v))
        vs = cache.vs.cpu().numpy()[cache.table[s, p // cache.ps], :, p % cache.ps // BLOCK].astype(np.float64)
        want, S, A, W = kv.attend(qh[s, :n], k, v, scale, seen, vs)
        d = 128 * 2.0 ** -24 * A
        if act == "bf16":
            R = q.shape[2] // k.shape[1]
            wide = np.abs(k).sum(-1).max(0) if len(k) else np.zeros(k.shape[1])
            d = d + 2.0 ** -17 * np.abs(qh[s, :n]).max(-1, keepdims=True) * abs(scale) * np.repeat(wide, R)[:, None]
            tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 1e-5 + 2 * d) * S
        else:
            tol = 2.0 ** -24 * np.abs(want) + (2.0 ** -21 + 1e-5 + 2 * (d + 2.0 ** -21 * A)) * S
        tol = tol + 2.0 ** (-25 if act == "bf16" else -40) * W + 2.0 ** -126 * (1 + np.repeat(np.abs(v).sum(0), q.shape[2] // v.shape[1], 0))
        err = np.abs(got[s, :n] - want)
        assert np.all(np.isfinite(got[s, :n]))
        assert np.all(err <= tol), (s, float((err - tol).max()), np.unravel_index((err - tol).argmax(), err.shape))
    return cache


ATTN_CASES = [
    # act, causal, ps, Hq, Hkv, lengths before, new
    ("bf16", True, 64, 40, 8, [0, 1, 14, 15, 16, 63, 64, 127, 300], [1] * 9),
    ("bf16", True, 16, 5, 1, [700, 0, 33, 2000], [1, 1, 0, 1]),
    ("bf16", True, 128, 16, 1, [257, 64], [1, 1]),
    ("bf16", True, 32, 8, 8, [100, 31, 95], [1, 1, 1]),
    ("bf16", True, 64, 10, 2, [61, 0, 130], [3, 2, 3]),
    ("bf16", True, 32, 40, 8, [77, 0, 5, 128], [9, 23, 0, 16]),
    ("bf16", True, 16, 5, 1, [0, 40], [130, 77]),
    ("bf16", True, 128, 2, 2, [3, 300], [200, 257]),
    ("bf16", True, 64, 12, 1, [1500], [40]),
    ("bf16", True, 64, 130, 1, [90], [2]),
    ("bf16", False, 64, 10, 2, [0, 1, 65, 300], [3, 1, 2, 0]),
    ("bf16", False, 16, 40, 8, [251, 0, 16], [33, 40, 7]),
    ("bf16", False, 128, 8, 4, [500, 129], [1, 1]),
    # many kv heads: the form for many rows
    ("bf16", True, 32, 160, 32, [77, 0, 5, 128], [9, 23, 0, 16]),
    ("bf16", True, 16, 160, 32, [0, 40], [130, 77]),
    ("bf16", True, 128, 32, 32, [3, 300], [200, 257]),
    ("bf16", True, 64, 96, 8, [1500], [40]),
    ("bf16", True, 64, 4160, 32, [90], [2]),
    ("bf16", False, 16, 160, 32, [251, 0, 16], [33, 40, 7]),
    ("f32", True, 64, 12, 2, [0, 1, 63, 64, 500], [1] * 5),
    ("f32", True, 16, 5, 1, [0, 40, 17], [35, 17, 0]),
    ("f32", False, 32, 16, 2, [77, 0, 300], [9, 4, 1]),
]


@pytest.mark.parametrize("case", range(len(ATTN_CASES)))
def test_attention(m2, case):
    act, causal, ps, Hq, Hkv, lengths, new = ATTN_CASES[case]
    S, T = len(lengths), max(new)
    reach = [L + n if causal else L for L, n in zip(lengths, new)]
    cache = _fill(m2, 100 + case, S, Hkv, ps, act, reach, capacity=max(reach) + 40)
    q, _ = _rows(7 + case, S, T, Hq, act)
    got = cache.attend(q, causal, _int(new), lengths=_int(lengths), pad=8 * (case % 2))
    _check(cache, q, got, lengths, new, causal, D ** -0.5, act)
    assert m2.mamba2_device_error() == 0


@pytest.mark.parametrize("T", [1, 24, 200])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_long_cache_split_over_the_gpu(m2, act, T):
    """One session, thousands of positions: the work along the cache is split
    and joined; n_new NULL."""
    L, ps = 5003, 64
    cache = _fill(m2, 11, 1, 2, ps, act, [L + T])
    q, _ = _rows(12, 1, T, 6, act)
    got = cache.attend(q, True, None, lengths=_int([L]))
    _check(cache, q, got, [L], [T], True, D ** -0.5, act)


@pytest.mark.parametrize("S", [80, 200])
def test_more_sessions_than_the_gpu_holds(m2, S):
    """Single frames of many sessions of all lengths, some equal, some empty,
    some without a new position: the order in which they run is not theirs."""
    rng = np.random.default_rng(S)
    lengths = [int(x) for x in rng.choice([0, 1, 17, 60, 64, 65, 130], S)]
    new = [int(x) for x in rng.choice([1, 1, 1, 0], S)]
    Hkv = 4 if S == 80 else 2
    cache = _fill(m2, 91, S, Hkv, 16, "bf16", [L + n for L, n in zip(lengths, new)])
    q, _ = _rows(92, S, 1, 3 * Hkv, "bf16")
    got = cache.attend(q, True, _int(new), lengths=_int(lengths))
    _check(cache, q, got, lengths, new, True, D ** -0.5, "bf16")
    got = cache.attend(q, False, _int(new), lengths=_int(lengths))
    _check(cache, q, got, lengths, new, False, D ** -0.5, "bf16")


@pytest.mark.parametrize("T,Hkv", [(2, 1), (40, 1), (40, 64)])
def test_uneven_scales_and_large_scores(m2, T, Hkv):
    """Values of some blocks a million times smaller or all zero, queries that
    make one position nearly everything, a negative scale, zero queries."""
    act, S, L, ps = "bf16", 1, 150, 32
    cache = Cache(m2, S, Hkv, ps, L + T, act)
    (k, _), (v, _) = _rows(21, S, L + T, Hkv, act), _rows(22, S, L + T, Hkv, act)
    v[0, 0:16] *= 2.0 ** -20
    v[0, 16:32] = 0
    v[0, 64:80] *= 2.0 ** 12
    v[0, 80:96] = 0
    k[0, 96:112] *= 2.0 ** -30
    cache.append(k, v)
    q, _ = _rows(23, S, T, 4 * Hkv, act)
    q[0, :, 0] = k[0, 3, 0] * 4   # position 3 (tiny values) nearly alone
    q[0, :, 1] = k[0, 20, 0] * 4  # position 20 (zero values) nearly alone
    q[0, :, 2] = 0
    for scale in (D ** -0.5, -0.05, 0.0):
        got = cache.attend(q, True, None, scale=scale, lengths=_int([L]))
        _check(cache, q, got, [L], [T], True, scale, act)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("T,Hkv", [(9, 1), (80, 1), (80, 32)])
def test_a_block_that_is_not_finite_reaches_only_who_sees_it(m2, T, Hkv, bad):
    """NaN or infinite values (and keys) in a block of the new positions: the
    queries before it are right, those that see it are NaN; its session alone."""
    import torch
    act, S, L, ps = "bf16", 2, 43, 16
    first = (L + T - 1) // BLOCK * BLOCK  # the last block's first position
    for where in "kv":
        cache = Cache(m2, S, Hkv, ps, L + T, act)
        rows = {n: _rows(95, S, L + T, Hkv, act)[0] for n in "kv"}
        rows[where][1, L + T - 1, 0, 5] = bad
        cache.append(rows["k"], rows["v"])
        q, _ = _rows(96, S, T, 5 * Hkv, act)
        got = cache.attend(q, True, None, lengths=_int([L, L]))
        good = first - L  # queries of session 1 that end before the block
        assert 0 < good < T
        new = [T, good]
        assert not bool(torch.isnan(got[:, :, 5:]).any())  # the other kv heads
        part = got.clone()
        part[1, good:] = -7.0
        _check(cache, q, part, [L, L], new, True, D ** -0.5, act)
        assert bool(torch.isnan(got[1, good:, :5]).any(-1).all())
        assert m2.mamba2_device_error() == 0


@pytest.mark.parametrize("act,T", [("bf16", 1), ("bf16", 8), ("bf16", 60), ("bf16", 500), ("f32", 6)])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_query_that_is_not_finite_reaches_only_its_row(m2, act, T, bad):
    """An infinity or a NaN in one head of one query gives that row NaN (its
    softmax has no value), and leaves every other row of the call right; where
    the row sees nothing it is zeros."""
    import torch
    Hkv, R, L = 2, 5, 77
    cache = _fill(m2, 97, 2, Hkv, 32, act, [L + T] * 2)
    q, _ = _rows(98, 2, T, Hkv * R, act)
    clean = cache.attend(q, True, None, lengths=_int([L, L])).clone()
    dirty = q.clone()
    dirty[1, T - 1, 3, 17] = bad
    got = cache.attend(dirty, True, None, lengths=_int([L, L]))
    assert bool(torch.isnan(got[1, T - 1, 3]).all())
    got[1, T - 1, 3] = clean[1, T - 1, 3]
    assert torch.equal(got, clean)
    assert not bool(cache.attend(dirty, False, None, lengths=_int([0, 0])).any())
    assert m2.mamba2_device_error() == 0


@pytest.mark.parametrize("T", [1, 30, 700])
def test_refused_sessions(m2, T):
    """A negative length, positions past the page table, a page outside the
    pool: the error word tells, the other sessions are right, and a refused
    append leaves its session as it was."""
    import torch
    act, Hkv, ps, L = "bf16", 2, 32, 50
    cache = _fill(m2, 31, 4, Hkv, ps, act, [L + T] * 4)
    q, _ = _rows(32, 4, T, 4, act)
    cap = cache.columns * ps
    got = cache.attend(q, True, None, lengths=_int([L, -1, cap - T + 1, L]))
    assert m2.mamba2_device_error() == 0x104
    g = got.float().cpu()
    assert torch.all(g[1] == 0) and torch.all(g[2] == 0)
    _check(cache, q[[0]], got[[0]], [L], [T], True, D ** -0.5, act)
    before = cache.host()
    k, _ = _rows(33, 4, T, Hkv, act)
    cache.append(k, k, None, lengths=_int([-5, cap, cap - T + 1, 2 ** 31 - 1]))
    assert m2.mamba2_device_error() == 0x104
    for a, b in zip(before, cache.host()):
        _same(a, b)
    rope, _, _ = _rope(m2, 64, L, False)  # a rotation table that ends too early
    cache.append(k, k, None, rope, lengths=_int([L] * 4))
    assert m2.mamba2_device_error() == 0x104
    cache.d_table[2, 0] = cache.n_pages
    cache.d_table[3, 0] = -1
    got = cache.attend(q, True, None, lengths=_int([L] * 4))
    assert m2.mamba2_device_error() == 0x105
    _check(cache, q[[0]], got[[0]], [L], [T], True, D ** -0.5, act)
    cache.append(k, k, None, lengths=_int([L, L, 0, 0]))
    assert m2.mamba2_device_error() == 0x105


def test_frames_as_they_are_used(m2):
    """A prompt, then single frames, each appended and attended: every frame's
    outputs are right for the cache at that time (the open block's scale may
    still grow), and the cache ends with the bits that one prefill leaves. The
    frame's two calls are captured in a graph and replayed with the lengths
    advancing on the device."""
    import torch
    act, S, Hq, Hkv, ps, prompt, frames = "bf16", 2, 10, 2, 16, 21, 30
    n = prompt + frames
    rope = _rope(m2, 128, n, False)[0]
    (k, _), (v, _), (q, _) = _rows(41, S, n, Hkv, act), _rows(42, S, n, Hkv, act), _rows(43, S, n, Hq, act)
    whole = Cache(m2, S, Hkv, ps, n, act, seed=1)
    qr = whole.append(k, v, None, rope, q)
    want = whole.attend(qr)
    steps = Cache(m2, S, Hkv, ps, n, act, seed=2)
    steps.append(k[:, :prompt], v[:, :prompt], None, rope)
    steps.lengths += prompt
    kv_row = torch.empty(S, 1, 2 * Hkv * D, dtype=torch.bfloat16, device="cuda")
    q_row, q_rot = (torch.empty(S, 1, Hq * D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    out = torch.empty_like(q_row)
    ws = torch.empty(max(1, m2.mamba2_attn_paged_workspace_bytes(steps.desc, 1, Hq)), dtype=torch.uint8, device="cuda")

    def frame():
        m2.mamba2_kv_append(steps.desc, 1, steps.lengths, None, kv_row, kv_row[0, 0, Hkv * D:], 2 * Hkv * D, rope, Hq, q_row,
                            Hq * D, q_rot, Hq * D)
        m2.mamba2_attn_paged(steps.desc, 1, Hq, True, steps.lengths, None, q_rot, Hq * D, D ** -0.5, out, Hq * D, ws)
        steps.lengths.add_(1)

    graph = None
    for t in range(prompt, n):
        kv_row[:, 0] = torch.cat((k[:, t].reshape(S, -1), v[:, t].reshape(S, -1)), -1)
        q_row[:, 0] = q[:, t].reshape(S, -1)
        if t < prompt + 2:
            frame()
        else:
            if graph is None:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    frame()
            graph.replay()
        _check(steps, q_rot.view(S, 1, Hq, D), out.view(S, 1, Hq, D), [t] * S, [1] * S, True, D ** -0.5, act)
        assert torch.equal(q_rot.view(S, Hq, D), qr[:, t])
    for s in range(S):
        for x, y in zip(whole.read(s, n), steps.read(s, n)):
            _same(x, y)
    _check(whole, qr, want, [0] * S, [n] * S, True, D ** -0.5, act)


def test_shared_prefix_pages(m2):
    """Two sessions list the same pages of a common prefix."""
    act, Hkv, ps = "bf16", 1, 16
    cache = _fill(m2, 51, 2, Hkv, ps, act, [48, 48])
    cache.table[1, :2] = cache.table[0, :2]
    cache.d_table.copy_(_int(cache.table.tolist()))
    q, _ = _rows(52, 2, 1, 4, act)
    got = cache.attend(q, True, None, lengths=_int([47, 47]))
    _check(cache, q, got, [47, 47], [1, 1], True, D ** -0.5, act)


def test_pool_past_32_bit_offsets(m2):
    """A pool of more than 4 GiB of keys, used at its far end."""
    import torch
    act, Hkv, ps, T = "bf16", 8, 128, 200
    n_pages = (1 << 32) // (Hkv * ps * D) + 40
    cache = Cache(m2, 1, Hkv, ps, T, act)
    cache.n_pages, cache.columns = n_pages, 2
    cache.table = np.array([[n_pages - 1, n_pages - 3]], np.int32)
    cache.d_table = torch.from_numpy(cache.table).cuda()
    cache.kp, cache.vp = (torch.zeros(n_pages, Hkv, ps, D, dtype=torch.uint8, device="cuda") for _ in "kv")
    cache.ks, cache.vs = (torch.ones(n_pages, Hkv, ps // BLOCK, device="cuda") for _ in "kv")
    cache.desc = m2.kv_cache(1, Hkv, ps, n_pages, 2, cache.d_table, cache.kp, cache.vp, cache.ks, cache.vs, cache.kt,
                             cache.vt, act=act)
    (k, kh), (v, vh) = _rows(61, 1, T, Hkv, act), _rows(62, 1, T, Hkv, act)
    cache.append(k, v)
    codes, scales = kv.quantise(kh[0])
    p = np.arange(T)
    far = cache.kp[n_pages - 4:].cpu().numpy()
    np.testing.assert_array_equal(far[np.where(p < ps, 3, 1), :, p % ps], codes)
    assert int(cache.kp[:n_pages - 4].max()) == 0 and m2.mamba2_device_error() == 0
    for n in (1, 40, T):
        q, _ = _rows(63, 1, n, 40, act)
        got = cache.attend(q, True, None, lengths=_int([T - n]))
        small = Cache(m2, 1, Hkv, ps, T, act)
        small.append(k, v)
        _check(small, q, got, [T - n], [n], True, D ** -0.5, act)


@pytest.mark.parametrize("T", [20, 400])
def test_two_streams_with_their_own_workspaces(m2, T):
    import torch
    act, Hkv, ps = "bf16", 2, 64
    caches = [_fill(m2, 70 + i, 1, Hkv, ps, act, [900 + T]) for i in range(2)]
    qs = [_rows(72 + i, 1, T, 8, act)[0] for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for c, q, st in zip(caches, qs, streams):
        with torch.cuda.stream(st):
            got.append(c.attend(q, True, None, lengths=_int([900])))
    torch.cuda.synchronize()
    for c, q, g in zip(caches, qs, got):
        _check(c, q, g, [900], [T], True, D ** -0.5, act)


def test_the_same_call_gives_the_same_bits(m2):
    import torch
    for T, L in ((1, 3000), (33, 2000), (300, 0), (1000, 2000)):
        cache = _fill(m2, 80, 1, 1, 32, "bf16", [L + T])
        q, _ = _rows(81, 1, T, 5, "bf16")
        a = cache.attend(q, True, None, lengths=_int([L])).clone()
        b = cache.attend(q, True, None, lengths=_int([L]))
        assert torch.equal(a, b)


@pytest.mark.parametrize("act,S,T,Hq,Hkv,longest", [
    ("bf16", 30, 1, 24, 8, 2000),   # frames, two CTAs and more to a session, more than the GPU holds
    ("bf16", 5, 3, 40, 8, 4000),    # 15 rows, eight and more CTAs
    ("f32", 9, 2, 12, 2, 2047),
    ("bf16", 6, 75, 40, 8, 1500),   # tiles, shared by two CTAs
    ("bf16", 2, 75, 40, 8, 2500),   # ... by four
    ("bf16", 2, 300, 10, 2, 700),   # long runs of rows whose tiles see different numbers of positions
])
def test_sessions_of_very_different_ages(m2, act, S, T, Hq, Hkv, longest):
    """Work along the cache shared by clusters where the sessions' lengths
    differ: some of a cluster's CTAs have nothing, or see nothing."""
    rng = np.random.default_rng(S * 1000 + T)
    lengths = [longest, 0] + [int(x) for x in rng.integers(0, longest, S - 2)]
    new = [T, T] + [int(x) for x in rng.integers(0, T + 1, S - 2)]
    cache = _fill(m2, 201, S, Hkv, 32, act, [L + n for L, n in zip(lengths, new)])
    q, _ = _rows(202, S, T, Hq, act)
    for causal in (True, False):
        got = cache.attend(q, causal, _int(new), lengths=_int(lengths))
        _check(cache, q, got, lengths, new, causal, D ** -0.5, act)
    assert m2.mamba2_device_error() == 0


def test_calls_from_two_threads(m2):
    """Two host threads, each with its own cache and stream, at once."""
    import threading

    import torch
    act, Hkv, ps = "bf16", 2, 64
    work = []
    for i, (T, L) in enumerate(((1, 500), (400, 900))):
        cache = _fill(m2, 211 + i, 1, Hkv, ps, act, [L + T])
        work.append((cache, _rows(213 + i, 1, T, 8, act)[0], L, T, torch.cuda.Stream()))
    torch.cuda.synchronize()
    got, failed = [None, None], []

    def run(i):
        cache, q, L, T, stream = work[i]
        try:
            with torch.cuda.stream(stream):
                for _ in range(30):
                    got[i] = cache.attend(q, True, None, lengths=_int([L]))
                stream.synchronize()
        except Exception as e:  # noqa: BLE001 (reported by the main thread)
            failed.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for i, (cache, q, L, T, _) in enumerate(work):
        _check(cache, q, got[i], [L], [T], True, D ** -0.5, act)
