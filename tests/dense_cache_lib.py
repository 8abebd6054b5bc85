"""What the GPU tests of the bounded dense caches share: caches and packed rows
on the GPU, with NaN wherever nothing was put, and the bounds of their checks.

With u = 2^-24, A a row's largest |scale| sum |q| |k| and mag = sum_p softmax_p |v_p|:
  scores   an fp32 sum of 128 products in any order is off by at most 128 u A,
           and its product with scale log2(e), the difference to a maximum (at
           most A log2(e) itself) and the rounded factor by 4 u A more:
           d = 132 u A. Times 2^x, a weight moves by d of itself.
  weights  exp2 to 2^-22 of itself and fp32 sums of a few thousand positive
           terms, in parts of at most some hundred: 1e-5 of the sum. In bf16 a
           weight enters its product with the values rounded: 2^-8 of itself.
  out      so (2 d + 1e-5 [+ 2^-8]) mag, and one rounding, 2^-8 |out| in bf16
           and 2^-24 in fp32; 2^-126 for what lies below the normal numbers.
  lse      d + 1e-5 + 4 u |lse|.
  sums     a weight e^(a - lse), with lse given: d + 4 u (A + |lse|) of itself for
           the exponent, and 1e-5 of the sum as above; the sum with the old one
           once more 2 u.
"""
import math

import numpy as np

from oracle import dense_cache as dc

D = dc.D
U = 2.0 ** -24


def dtype(act):
    import torch
    return torch.bfloat16 if act == "bf16" else torch.float32


def score_bound(size):
    return 132 * U * size


class Caches:
    """Dense caches of sessions with `before` positions each; NaN past them."""

    def __init__(self, m2, before, Hq, Hkv, act, max_len, seed=0, spread=1.0):
        import torch
        self.m2, self.Hq, self.Hkv, self.act, self.max_len = m2, Hq, Hkv, act, max_len
        self.before, self.S = list(before), len(before)
        g = torch.Generator().manual_seed(seed)
        self.g, self.spread = g, spread
        self.kc, self.vc = (torch.full((self.S, Hkv, max_len, D), math.nan, dtype=dtype(act), device="cuda") for _ in "kv")
        for s, b in enumerate(before):
            if 0 < b <= max_len:
                self.kc[s, :, :b] = self.values(Hkv, b, D)
                self.vc[s, :, :b] = self.values(Hkv, b, D)
        self.lengths = torch.tensor(self.before, dtype=torch.int32, device="cuda")

    def values(self, *shape):
        import torch
        return (torch.randn(*shape, generator=self.g) * self.spread).to(dtype(self.act)).cuda()

    def host(self, s, n):
        return [x[s, :, :n].double().cpu().numpy() for x in (self.kc, self.vc)]


class Packed:
    """Packed q | k | v rows: sessions of `new` rows behind `lead` rows that
    belong to none, `tail` of them at the end; both NaN."""

    def __init__(self, c, new, lead=0, tail=0, pad=0):
        import torch
        self.c, self.new = c, list(new)
        starts = np.concatenate([[0], np.cumsum(new)]) + lead
        self.starts = starts.tolist()
        self.n_rows = int(starts[-1]) + tail
        Hq, Hkv = c.Hq, c.Hkv
        self.width = (Hq + 2 * Hkv) * D + pad
        self.rows = torch.full((max(1, self.n_rows), self.width), math.nan, dtype=dtype(c.act), device="cuda")
        if sum(new):
            self.rows[lead:int(starts[-1]), :self.width - pad] = c.values(sum(new), self.width - pad)
        self.q, self.k, self.v = self.rows[:, :Hq * D], self.rows[:, Hq * D:(Hq + Hkv) * D], self.rows[:, (Hq + Hkv) * D:]
        self.row_start = torch.tensor(self.starts, dtype=torch.int32, device="cuda")
        self.out_width = Hq * D + pad
        self.out = torch.full((max(1, self.n_rows), self.out_width), -7.0, dtype=dtype(c.act), device="cuda")
        self.lse = torch.full((max(1, self.n_rows), Hq), -7.0, device="cuda")

    def attend(self, scale=D ** -0.5, lse=True, lengths="own", stream=None, row_start=None):
        c = self.c
        self.scale = scale
        c.m2.mamba2_attn_prompt(c.S, self.n_rows, c.Hq, c.Hkv, D, c.max_len, c.act,
                                self.row_start if row_start is None else row_start,
                                c.lengths if isinstance(lengths, str) else lengths, self.q, self.width, self.k, self.v,
                                self.width, c.kc, c.vc, scale, self.out, self.out_width, self.lse if lse else None,
                                stream=stream)

    def weigh(self, acc, acc_out, window, stream=None, row_start=None):
        c = self.c
        c.m2.mamba2_attn_prompt_weights(c.S, self.n_rows, c.Hq, c.Hkv, D, c.max_len, c.act,
                                        self.row_start if row_start is None else row_start, c.lengths, self.q, self.width,
                                        c.kc, self.scale, self.lse, window, acc, acc_out, stream=stream)

    def mine(self, s):
        return slice(self.starts[s], self.starts[s + 1])

    def check(self, sessions=None, lse=True, rows=None):
        """out, lse and the caches of the sessions (all) against fp64, with their
        new rows in the caches bit for bit; nothing else written."""
        import torch
        c = self.c
        every = range(c.S) if sessions is None else sessions
        untouched = np.ones(max(1, self.n_rows), bool)
        for s in every:
            b, n = c.before[s], self.new[s]
            untouched[self.mine(s)] = False
            if n:
                for cache, new in ((c.kc, self.k), (c.vc, self.v)):
                    want = new[self.mine(s), :c.Hkv * D].reshape(n, c.Hkv, D).transpose(0, 1)
                    assert torch.equal(cache[s, :, b:b + n].view(torch.uint8), want.contiguous().view(torch.uint8))
            assert torch.isnan(c.kc[s, :, b + n:]).all() and torch.isnan(c.vc[s, :, b + n:]).all()
            if n == 0:
                continue
            k, v = c.host(s, b + n)
            q = self.q[self.mine(s)].double().cpu().numpy().reshape(n, c.Hq, D)
            check_rows(self.out[self.mine(s), :c.Hq * D].double().cpu().numpy().reshape(n, c.Hq, D),
                       self.lse[self.mine(s)].double().cpu().numpy() if lse else None, q, k, v, self.scale, b, c.act)
        left = torch.from_numpy(untouched).cuda()
        if sessions is None:
            assert torch.all(self.out[left] == -7) and torch.all(self.lse[left] == -7)
        assert torch.all(self.out[:, c.Hq * D:] == -7)
        if not lse:
            assert torch.all(self.lse == -7)


def check_rows(out, lse, q, k, v, scale, before, act):
    want, want_lse, mag, size = dc.attend(q, k, v, scale, before)
    d = score_bound(size)
    half = 2.0 ** -8 if act == "bf16" else U
    tol = (2 * d[..., None] + 1e-5 + (half if act == "bf16" else 0)) * mag + half * np.abs(want) + 2.0 ** -126
    worst = np.abs(out - want) / tol
    assert np.all(worst <= 1), f"out: {worst.max():.3g} of the bound"
    if lse is not None:
        worst = np.abs(lse - want_lse) / (d + 1e-5 + 4 * U * np.abs(want_lse))
        assert np.all(worst <= 1), f"lse: {worst.max():.3g} of the bound"


def check_sums(got, acc, q, k, scale, before, lse, window):
    """acc_out [Hkv, L] against acc [Hkv, before] and the rows' weights."""
    n = q.shape[0]
    want = dc.received(q, k, scale, before, lse, window)
    _, size = dc.scores(q, k, scale, before)
    first = max(0, n - window)
    exponent = score_bound(size[:, first:].max(initial=0.0)) + \
        4 * U * (size[:, first:].max(initial=0.0) + np.abs(lse[first:]).max(initial=0.0))
    tol = (exponent + 1e-5) * want
    want[:, :before] += acc[:, :before]
    tol += 2 * U * np.abs(want) + 2.0 ** -126
    worst = np.abs(got - want) / tol
    assert np.all(worst <= 1), f"sums: {worst.max():.3g} of the bound"
