"""The bounded dense caches at the edges of what their header allows. The bounds
stand in tests/dense_cache_lib.py; where a test has one of its own, it is derived
beside it."""
import math

import numpy as np
import pytest

from dense_cache_lib import D, Caches, Packed, check_rows, check_sums, dtype

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m2():
    import full_duplex_speech_gb300 as m2
    m2.load()
    m2.mamba2_device_error()
    return m2


def _done(m2, code=0):
    import torch
    torch.cuda.synchronize()
    assert m2.mamba2_device_error() == code


def _some_of(m2, c, p, sessions, seed=0):
    """The caches as they are now and the rows of some sessions alone."""
    import torch
    d = Caches(m2, [c.before[s] for s in sessions], c.Hq, c.Hkv, c.act, c.max_len, seed=seed)
    d.kc.copy_(c.kc[sessions]), d.vc.copy_(c.vc[sessions])
    q = Packed(d, [p.new[s] for s in sessions])
    q.rows.copy_(torch.cat([p.rows[p.mine(s)] for s in sessions]))
    return d, q


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_refused_sessions_among_many_pairs_of_tiles(m2, act):
    """Several pairs of tiles a CTA: long chunks' pairs whose second tile has no rows, and refused pairs of two
    tiles, in turn. What is not refused comes out as in a call without the others, bit for bit."""
    import torch
    kinds = [(700, 40), (-1, 32), (900, 8), (1024, 64)]
    b, n = ([k[i] for k in kinds * 40] for i in range(2))
    c = Caches(m2, b, 32, 4, act, 1024, seed=82)
    p = Packed(c, n)
    good = [s for s in range(160) if s % 2 == 0]
    d, q = _some_of(m2, c, p, good)
    q.attend()
    _done(m2)
    held = c.kc[1::2].clone(), c.vc[1::2].clone()
    for _ in range(10):
        p.out.fill_(-7.0), p.lse.fill_(-7.0)
        p.attend()
        _done(m2, 0x104)
        assert torch.equal(torch.cat([p.out[p.mine(s)] for s in good]), q.out)
        assert torch.equal(torch.cat([p.lse[p.mine(s)] for s in good]), q.lse)
    p.check(sessions=[0, 2, 78, 158])
    for s in range(1, 160, 2):
        assert torch.all(p.out[p.mine(s)] == 0) and torch.all(p.lse[p.mine(s)] == -math.inf)
    for now, was in zip((c.kc, c.vc), held):
        assert torch.equal(now[1::2].view(torch.uint8), was.view(torch.uint8))
    for now, want in ((c.kc, d.kc), (c.vc, d.vc)):
        assert torch.equal(now[::2].view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_negative_scales_over_many_pairs_of_tiles(m2, act):
    """Several pairs of tiles a CTA, some with one tile only: the scale's sign and the queries' are the same."""
    import torch
    b, n = [0, 300, 0, 500] * 40, [8, 40, 75, 16] * 40
    c = Caches(m2, b, 32, 4, act, 600, seed=83)
    p, q = Packed(c, n), Packed(c, n)
    q.rows.copy_(p.rows)
    q.q.neg_()
    q.attend(scale=0.11)
    _done(m2)
    for _ in range(10):
        p.out.fill_(-7.0), p.lse.fill_(-7.0)
        p.attend(scale=-0.11)
        _done(m2)
        assert torch.equal(p.out, q.out) and torch.equal(p.lse, q.lse)
    p.check(sessions=[0, 1, 2, 3, 157, 159])


def _own_rows(starts, n_rows):
    """Sessions whose rows lie within the call's and behind every entry ahead of their first."""
    return [s for s in range(len(starts) - 1)
            if 0 <= starts[s] <= starts[s + 1] <= n_rows and starts[s] >= max(starts[:s], default=0)]


def _long_row_starts(S, at, by):
    """Sessions of up to three rows, with one entry raised."""
    starts = np.concatenate([[0], np.cumsum(np.random.default_rng(S).integers(0, 4, S))])
    starts[at] += by
    return starts.tolist()


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("starts,n_rows", [
    ([0, 100, 50, 150], 150), ([0, 40, 30, 70], 70), ([0, 100, 50, 60, 150, 170], 170), ([0, 30, -1, 60], 60),
    ([10, 20, 500, 30, 60], 60), ([50, 0, 60, 80], 80), ([0, 0, 64, 63, 64, 128], 128),
    (_long_row_starts(200, 20, 40), 300), (_long_row_starts(900, 127, 3000), 1400), (_long_row_starts(900, 600, 100), 1400),
    (_long_row_starts(1100, 1024, 9), 1700),
])
def test_row_starts_that_decrease(m2, act, starts, n_rows):
    """The sessions on both sides, and those that begin before an entry ahead of them, are left out: their caches and
    sums, and rows that are nobody else's, stay as they were. The others come out as usual, theirs appended."""
    import torch
    S, Hq, Hkv, scale = len(starts) - 1, 10, 2, D ** -0.5
    good = _own_rows(starts, n_rows)
    assert good != list(range(S))
    b = [(7 * s) % 40 for s in range(S)]
    c = Caches(m2, b, Hq, Hkv, act, 160, seed=84)
    p = Packed(c, [n_rows] + [0] * (S - 1))
    row_start = torch.tensor(starts, dtype=torch.int32, device="cuda")
    was = c.kc.clone(), c.vc.clone()
    acc = torch.rand(S, Hkv, c.max_len, device="cuda")
    sums = torch.full_like(acc, -7.0)
    p.attend(row_start=row_start)
    _done(m2, 0x106)
    p.weigh(acc, sums, 5, row_start=row_start)
    _done(m2, 0x106)
    mine = torch.zeros(n_rows, dtype=torch.bool, device="cuda")
    for s in range(S):
        if s not in good:
            for now, old in zip((c.kc, c.vc), was):
                assert torch.equal(now[s].view(torch.uint8), old[s].view(torch.uint8))
            assert torch.all(sums[s] == -7)
            continue
        at, n = starts[s], starts[s + 1] - starts[s]
        mine[at:at + n] = True
        for cache, rows in ((c.kc, p.k), (c.vc, p.v)):
            want = rows[at:at + n, :Hkv * D].reshape(n, Hkv, D).transpose(0, 1).contiguous()
            assert torch.equal(cache[s, :, b[s]:b[s] + n].contiguous().view(torch.uint8), want.view(torch.uint8))
            assert torch.isnan(cache[s, :, b[s] + n:]).all()
        if S < 100 or s % 25 == 0 or s > S - 10:
            k, v = c.host(s, b[s] + n)
            q = p.q[at:at + n].double().cpu().numpy().reshape(n, Hq, D)
            lse = p.lse[at:at + n].double().cpu().numpy()
            if n:
                check_rows(p.out[at:at + n, :Hq * D].double().cpu().numpy().reshape(n, Hq, D), lse, q, k, v, scale, b[s], act)
            check_sums(sums[s, :, :b[s] + n].double().cpu().numpy(), acc[s].double().cpu().numpy(), q, k, scale, b[s], lse, 5)
            assert torch.all(sums[s, :, b[s] + n:] == -7)
    assert torch.all(p.out[~mine] == -7) and torch.all(p.lse[~mine] == -7)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("what", ["start", "length"])
@pytest.mark.parametrize("one_row", [199, 0])
def test_what_is_wrong_behind_the_last_rows_is_recorded(m2, act, what, one_row):
    """Sessions without rows far behind those that have them (or none has): one whose rows would end past the call's, or
    whose length is past its cache."""
    import torch
    S = 700
    b = [3] * S
    if what == "length":
        b[650] = 13
    c = Caches(m2, b, 5, 1, act, 12, seed=85)
    p = Packed(c, [1] * one_row + [0] * (S - one_row))
    starts = list(p.starts)
    if what == "start":
        starts[-1] = 500
    held = c.kc[one_row:].clone()
    p.attend(row_start=torch.tensor(starts, dtype=torch.int32, device="cuda"))
    _done(m2, 0x106 if what == "start" else 0x104)
    p.check(sessions=range(0, one_row, 20))
    assert torch.equal(c.kc[one_row:].view(torch.uint8), held.view(torch.uint8))


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,max_len,before", [
    (40, 8, 300, [0, 1, 63, 64, 200, 299]), (40, 8, 7500, [7499]), (10, 2, 7500, [700]), (9, 3, 160, [40, 130, 0]),
])
def test_frames_of_scores_far_below_zero(m2, act, Hq, Hkv, max_len, before):
    """Keys all alike, so that a position's weight is 1 / positions whatever the scores, which here lie near
    -4e33 (every position's score comes from the same products in the same order: equal bits)."""
    import torch
    c = Caches(m2, before, Hq, Hkv, act, max_len, seed=80)
    key = (1 + torch.rand(D, generator=c.g)).to(dtype(act)).cuda() * 1e16
    for s, b in enumerate(before):
        c.kc[s, :, :b] = key
    q = -(1 + torch.rand(c.S, Hq, D, generator=c.g)).to(dtype(act)).cuda() * 1e16
    k, v = key.expand(c.S, Hkv, D).contiguous(), c.values(c.S, Hkv, D)
    kc, vc = c.kc.clone(), c.vc.clone()
    acc = torch.zeros(c.S, Hkv, max_len, device="cuda")
    sums, out = torch.full_like(acc, -7.0), torch.full((c.S, Hq, D), -7.0, dtype=dtype(act), device="cuda")
    need = m2.mamba2_attn_decode_weights_workspace_bytes(c.S, Hq, Hkv, D, max_len, act)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    m2.mamba2_attn_decode_weights(c.S, Hq, Hkv, D, max_len, act, c.lengths, q, k, v, c.kc, c.vc, D ** -0.5, out, acc, sums, ws)
    plain = torch.empty_like(out)
    ws = torch.empty(max(1, m2.mamba2_attn_decode_workspace_bytes(c.S, Hq, Hkv, D, max_len, act)), dtype=torch.uint8,
                     device="cuda")
    m2.mamba2_attn_decode(c.S, Hq, Hkv, D, max_len, act, c.lengths, q, k, v, kc, vc, D ** -0.5, plain, ws)
    _done(m2)
    assert torch.equal(out, plain)
    for s, b in enumerate(before):
        # a weight and a sum of them are within 1e-5 of themselves (the scores' own error is the same for all)
        want = Hq // Hkv / (b + 1)
        assert torch.all((sums[s, :, :b + 1] - want).abs() <= 1e-5 * want) and torch.all(sums[s, :, b + 1:] == -7)
        values = c.vc[s, :, :b + 1].double()
        mean, mag = (x.mean(1).repeat_interleave(Hq // Hkv, 0) for x in (values, values.abs()))
        half = 2.0 ** -8 if act == "bf16" else 2.0 ** -24
        assert torch.all((out[s].double() - mean).abs() <= (1e-5 + (half if act == "bf16" else 0)) * mag + half * mean.abs())


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("before,new", [([20, 0], [150, 60]), ([2000], [30]), ([0], [1])])
def test_a_scale_of_zero_and_large_products(m2, act, before, new):
    """A score is 0, however large its products are (here some 1e37)."""
    c = Caches(m2, before, 8, 2, act, max(b + n for b, n in zip(before, new)), seed=81)
    p = Packed(c, new, lead=1)
    c.kc.mul_(1e18), p.q.mul_(1e18), p.k.mul_(1e18)
    p.attend(scale=0.0)
    _done(m2)
    p.check()


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("before,new", [([20], [150]), ([2000], [40]), ([0], [300])])
def test_keys_of_infinite_scores(m2, act, before, new):
    """A key whose score is -infinity has no weight, as one of -1e30 has none; one of +infinity makes what sees it NaN."""
    import torch
    b, n = before[0], new[0]
    at = n // 3  # the row that it comes with
    found = []
    for key in (1e30, math.inf):
        c = Caches(m2, before, 10, 2, act, b + n, seed=86)
        p = Packed(c, new)
        p.q.view(n, -1)[:, 3::D] = -1.0                  # dim 3 of every head
        p.q.view(n, -1)[:, 5 * D + 3::D] = 1.0           # of kv head 1's: the score is +infinity
        p.k[at, 3] = key
        p.k[at, D + 3] = 0.0 if key == 1e30 else math.inf
        p.attend()
        acc = torch.zeros(1, 2, b + n, device="cuda")
        sums = torch.full_like(acc, -7.0)
        p.weigh(acc, sums, n)
        _done(m2)
        found.append([p.out.float().view(n, 10, D), p.lse.clone(), sums])
    (out, lse, sums), (out_inf, lse_inf, sums_inf) = found
    assert torch.equal(out_inf[:, :5], out[:, :5]) and torch.equal(lse_inf[:, :5], lse[:, :5])
    assert torch.equal(sums_inf[:, 0], sums[:, 0]) and torch.all(sums[0, 0, b + at] == 0)
    assert torch.equal(out_inf[:at, 5:], out[:at, 5:]) and torch.equal(lse_inf[:at, 5:], lse[:at, 5:])
    assert torch.isnan(out_inf[at:, 5:]).all() and not torch.isfinite(lse_inf[at:, 5:]).any()
    assert not torch.isfinite(sums_inf[0, 1, b + at])


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_lse_and_sums_have_no_bias(m2, act):
    """Over many rows what is random in single scores averages out, and what is left is a bias. The tensor cores' sums of
    128 products are cut off toward zero: a score comes out too small by some share of 2^-23 of itself that lies between
    a third and all, and is multiplied by 1 + 2^-23. So at most two thirds of 2^-23 of the scores that count are left,
    which lie below 7 here on average (their lse is near 10, of 2048 positions): 5.6e-7 of the sums, and with 1e-7 for
    fp32 sums and the exponentials 7e-7. Without that factor it was 1.0e-6. The lse's mean error is that of the
    average score that counts, below 4: 3.2e-7 (without 5e-7 to 7e-7)."""
    import torch
    n, Hq, Hkv, scale = 2048, 10, 2, D ** -0.5
    c = Caches(m2, [0], Hq, Hkv, act, n, seed=87)
    p = Packed(c, [n])
    g = torch.Generator(device="cuda").manual_seed(88)
    wide = torch.randn(p.rows.shape[1] // D, D, generator=g, device="cuda").mul(0.5).exp().flatten()
    p.rows.mul_(wide).mul_(torch.randn(n, 1, generator=g, device="cuda").mul(0.3).exp())
    p.attend(scale=scale)
    q, k = (x.reshape(n, -1, D).double() for x in (p.q[:, :Hq * D], p.k[:, :Hkv * D]))
    score = torch.einsum("nhd,phd->hnp", q, k.repeat_interleave(Hq // Hkv, 1)) * scale
    score.masked_fill_(torch.arange(n, device="cuda") > torch.arange(n, device="cuda")[:, None], -math.inf)
    lse = torch.logsumexp(score, -1)
    assert ((p.lse.T.double() - lse).mean()).abs() <= 3.2e-7
    p.lse.copy_(lse.T)
    acc = torch.zeros(1, Hkv, n, device="cuda")
    sums = torch.full_like(acc, -7.0)
    p.weigh(acc, sums, n)
    _done(m2)
    want = torch.exp(score - p.lse.T.double()[..., None]).view(Hkv, -1, n, n).sum((1, 2))
    assert (sums[0] - want).norm() <= 7e-7 * want.norm()
