"""GPU parity of the bounded dense caches where work is shared or meets other
work: positions of few rows shared by a cluster's CTAs, rows of sessions beside
one another, calls on two streams at once, calls without rows. The bounds stand
in tests/dense_cache_lib.py."""
import math

import numpy as np
import pytest

from dense_cache_lib import D, Caches, Packed, check_sums, dtype
from oracle import dense_cache as dc

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


# few rows behind long caches: two, four and eight CTAs share a pair of tiles
FEW = [(40, 8, [7400], [75]), (5, 1, [7400], [75]), (5, 1, [7400], [1]), (16, 2, [5000], [30]), (40, 8, [3000], [300]),
       (10, 2, [900, 2000, 0], [60, 75, 75]), (4, 4, [1500, 10], [2, 140]), (8, 1, [130], [200])]


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("scale,times", [(D ** -0.5, 1.0), (-0.07, 1.0), (D ** -0.5, 30.0)])
@pytest.mark.parametrize("Hq,Hkv,before,new", FEW)
def test_few_rows_behind_long_caches(m2, act, scale, times, Hq, Hkv, before, new):
    """Negative scales too, and scores whose maxima differ by hundreds from part to part."""
    import torch
    c = Caches(m2, before, Hq, Hkv, act, max(b + n for b, n in zip(before, new)), seed=50)
    p = Packed(c, new, lead=1, tail=2)
    p.q.mul_(times)
    p.attend(scale=scale)
    acc = torch.rand(c.S, Hkv, c.max_len, device="cuda")
    out = torch.full_like(acc, -7.0)
    p.weigh(acc, out, 40)
    _done(m2)
    p.check()
    for s, (b, n) in enumerate(zip(before, new)):
        k, _ = c.host(s, b + n)
        q = p.q[p.mine(s)].double().cpu().numpy().reshape(n, Hq, D)
        check_sums(out[s, :, :b + n].double().cpu().numpy(), acc[s].double().cpu().numpy(), q, k, scale, b,
                   p.lse[p.mine(s)].double().cpu().numpy(), 40)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("at", [0, 10, 74])
def test_values_that_are_not_finite_behind_long_caches(m2, act, at):
    import torch
    outs = []
    for bad in (False, True):
        c = Caches(m2, [2000], 5, 1, act, 2075, seed=51)
        p = Packed(c, [75])
        if bad:
            p.v[at, 9] = math.inf
        p.attend()
        _done(m2)
        outs.append((p.out.clone(), p.lse.clone()))
    (clean, lse), (out, lse_bad) = outs
    assert torch.equal(out[:at], clean[:at]) and torch.equal(lse, lse_bad)
    assert not torch.isfinite(out[at:].view(-1, 5, D)[:, :, 9]).any()


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_a_refused_session_behind_a_long_cache(m2, act):
    import torch
    c = Caches(m2, [7401], 5, 1, act, 7475, seed=52)
    p = Packed(c, [75])
    held = c.kc.clone()
    p.attend()
    _done(m2, 0x104)
    assert torch.all(p.out == 0) and torch.all(p.lse == -math.inf)
    assert torch.equal(c.kc.view(torch.uint8), held.view(torch.uint8))


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("before", [0, 6])
def test_what_is_not_finite_stays_in_its_session(m2, act, before):
    """Rows of the sessions on both sides, in the same tiles' copies, are all NaN or infinite."""
    import torch
    outs = []
    for bad in (False, True):
        c = Caches(m2, [before] * 3, 10, 2, act, 300, seed=53)
        p = Packed(c, [40, 131, 77])
        if bad:
            p.rows[:40], p.rows[171:] = math.nan, math.inf
        p.attend()
        acc = torch.zeros(3, 2, 300, device="cuda")
        sums = torch.full_like(acc, -7.0)
        p.weigh(acc, sums, 1000)
        _done(m2)
        outs.append([t.clone() for t in (p.out[40:171], p.lse[40:171], sums[1], c.kc[1].view(torch.uint8))])
    for now, want in zip(*outs):
        assert torch.equal(now, want)


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_many_pairs_of_tiles(m2, act):
    """Some hundred CTAs' worth of pairs, fresh sessions and such behind caches in turn."""
    rng = np.random.default_rng(54)
    n = rng.integers(0, 200, 60).tolist()
    b = [int(x) if i % 3 else 0 for i, x in enumerate(rng.integers(0, 300, 60))]
    c = Caches(m2, b, 40, 8, act, 500, seed=54)
    p = Packed(c, n)
    p.attend()
    _done(m2)
    p.check(sessions=range(0, 60, 5))


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_calls_without_rows(m2, act):
    """No rows in all: a prompt does nothing, and the sums so far are those."""
    import torch
    c = Caches(m2, [0, 37, 300], 10, 2, act, 300, seed=55)
    p = Packed(c, [0, 0, 0])
    held = c.kc.clone()
    p.attend()
    acc = torch.rand(3, 2, 300, device="cuda")
    out = torch.full_like(acc, -7.0)
    p.weigh(acc, out, 1000)
    _done(m2)
    assert torch.equal(c.kc.view(torch.uint8), held.view(torch.uint8)) and torch.all(p.out == -7)
    for s, b in enumerate(c.before):
        assert torch.equal(out[s, :, :b], acc[s, :, :b]) and torch.all(out[s, :, b:] == -7)


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_two_streams_at_once(m2, act):
    """A prompt, its weights, a frame and an eviction on each of two streams give what each gives alone."""
    import torch

    class Chain:
        def __init__(self, seed, Hq, Hkv, before, new):
            self.c = Caches(m2, before, Hq, Hkv, act, 1200, seed=seed)
            self.p = Packed(self.c, new)
            self.start = [t.clone() for t in (self.c.kc, self.c.vc)]
            S = len(before)
            self.acc0 = torch.rand(S, Hkv, 1200, device="cuda")
            self.acc = self.acc0.clone()
            self.then = self.c.lengths + torch.tensor(new, dtype=torch.int32, device="cuda")
            self.after = self.then + 1
            self.q, self.k, self.v = self.c.values(S, Hq, D), self.c.values(S, Hkv, D), self.c.values(S, Hkv, D)
            self.o = torch.empty(S, Hq, D, dtype=dtype(act), device="cuda")
            need = m2.mamba2_attn_decode_weights_workspace_bytes(S, Hq, Hkv, D, 1200, act)
            self.ws = torch.empty(need, dtype=torch.uint8, device="cuda")
            self.small = [torch.zeros(S, Hkv, 200, D, dtype=dtype(act), device="cuda") for _ in "kv"] + \
                [torch.zeros(S, Hkv, 200, device="cuda")]

        def reset(self):
            for t, was in zip((self.c.kc, self.c.vc, self.acc), self.start + [self.acc0]):
                t.copy_(was)
            for t in [self.p.out, self.p.lse, self.o] + self.small:
                t.zero_()

        def run(self, stream):
            c, S = self.c, self.c.S
            self.p.attend(stream=stream)
            self.p.weigh(self.acc, self.acc, 50, stream=stream)
            m2.mamba2_attn_decode_weights(S, c.Hq, c.Hkv, D, 1200, act, self.then, self.q, self.k, self.v, c.kc, c.vc, 0.1,
                                          self.o, self.acc, self.acc, self.ws, stream=stream)
            m2.mamba2_kv_evict(S, c.Hkv, D, 1200, act, self.after, c.kc, c.vc, self.acc, 200, 30, 200, *self.small, None,
                               stream=stream)
            m2.mamba2_kv_evict(S, c.Hkv, D, 1200, act, self.after, c.kc, c.vc, self.acc, 300, 50, 1200, c.kc, c.vc, self.acc,
                               None, stream=stream)

        def results(self):
            return [t.clone() for t in [self.c.kc, self.c.vc, self.acc, self.p.out, self.p.lse, self.o] + self.small]

    chains = [Chain(56, 40, 8, [900, 0, 31], [70, 600, 1]), Chain(57, 10, 2, [1100], [90])]
    streams = [torch.cuda.Stream() for _ in chains]
    want = []
    for ch in chains:
        ch.run(torch.cuda.current_stream())
        _done(m2)
        want.append(ch.results())
    for _ in range(5):
        for ch in chains:
            ch.reset()
        torch.cuda.synchronize()
        for ch, stream in zip(chains, streams):
            ch.run(stream)
        _done(m2)
        for ch, held in zip(chains, want):
            for now, was in zip(ch.results(), held):
                assert torch.equal(now.contiguous().view(torch.uint8), was.contiguous().view(torch.uint8))


@pytest.mark.parametrize("act,lead", [("f32", 240000), ("bf16", 300000)])
def test_rows_past_32_bits(m2, act, lead):
    """Rows of more than 2^31 elements, the sessions' at their end; nothing before them is written."""
    import torch
    c = Caches(m2, [33, 0], 40, 8, act, 100, seed=59)
    width = 56 * D + (2048 if act == "f32" else 0)
    assert lead * width > 2 ** 31
    p = Packed(c, [60, 21], lead=lead, pad=width - 56 * D)
    p.attend()
    acc = torch.rand(2, 8, 100, device="cuda")
    out = torch.full_like(acc, -7.0)
    p.weigh(acc, out, 1000)
    _done(m2)
    p.check()
    k, _ = c.host(0, 93)
    q = p.q[p.mine(0)].double().cpu().numpy().reshape(60, 40, D)
    check_sums(out[0, :, :93].double().cpu().numpy(), acc[0].double().cpu().numpy(), q, k, p.scale, 33,
               p.lse[p.mine(0)].double().cpu().numpy(), 1000)


@pytest.mark.parametrize("S,max_len,lens", [(1, 30000, [29999]), (3, 27000, [27000, 24577, 24576])])
def test_evictions_from_caches_longer_than_the_staged_keys(m2, S, max_len, lens):
    """Into smaller caches, by many CTAs a head; ties across the runs of positions."""
    import torch
    g = torch.Generator().manual_seed(58)
    k, v = (torch.randn(S, 2, max_len, D, generator=g).to(torch.bfloat16).cuda() for _ in "kv")
    acc = (torch.randint(0, 50, (S, 2, max_len), generator=g).float() / 8).cuda()
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ko, vo = (torch.full((S, 2, 9000, D), -7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    ao, kept = torch.full((S, 2, 9000), -7.0, device="cuda"), torch.full((S, 2, 8191), -7, dtype=torch.int32, device="cuda")
    m2.mamba2_kv_evict(S, 2, D, max_len, "bf16", lengths, k, v, acc, 8191, 999, 9000, ko, vo, ao, kept)
    _done(m2)
    for s in range(S):
        for h in range(2):
            stay = dc.kept(acc[s, h, :lens[s]].tolist(), 8191, 999)
            at = torch.tensor(stay, device="cuda")
            assert torch.equal(kept[s, h], at.int())
            for now, was in ((ko, k), (vo, v), (ao, acc)):
                assert torch.equal(now[s, h, :8191], was[s, h, at]) and torch.all(now[s, h, 8191:] == -7)


LENGTHS = [1, 2, 25, 26, 49, 50, 51, 75, 76, 100, 101, 127, 128, 129, 130, 255, 256, 257, 300]


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hkv", [(40, 8), (8, 8), (64, 8), (16, 8), (24, 8)])
@pytest.mark.parametrize("behind", [False, True])
def test_lengths_of_many_sessions(m2, act, Hq, Hkv, behind):
    """So many that a CTA takes a pair of tiles: the lengths around the edges of tiles, pairs and chunks."""
    before = [(37 * i) % 260 if behind else 0 for i in range(len(LENGTHS))]
    c = Caches(m2, before, Hq, Hkv, act, 600, seed=71)
    p = Packed(c, LENGTHS, lead=3, tail=2)
    p.attend()
    _done(m2)
    p.check()


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("place", [0, 0.5, 0.9])
@pytest.mark.parametrize("what", [math.nan, math.inf])
def test_values_that_are_not_finite_in_many_sessions(m2, act, place, what):
    """One value of each session; the rows that do not see it keep their bits, and the caches have it."""
    import torch
    outs = []
    for bad in (False, True):
        c = Caches(m2, [(41 * i) % 200 for i in range(len(LENGTHS))], 40, 8, act, 600, seed=72)
        p = Packed(c, LENGTHS)
        at = [p.starts[s] + int(place * (n - 1)) for s, n in enumerate(LENGTHS)]
        if bad:
            for row in at:
                p.v[row, 2 * D + 5] = what  # kv head 2
        p.attend()
        _done(m2)
        outs.append((p.out.view(-1, 40, D).clone(), p.lse.clone()))
    (clean, lse), (out, lse_bad) = outs
    assert torch.equal(lse, lse_bad)
    assert torch.equal(out[:, :10], clean[:, :10]) and torch.equal(out[:, 15:], clean[:, 15:])
    for s, n in enumerate(LENGTHS):
        b = c.before[s]
        assert torch.equal(out[p.starts[s]:at[s], 10:15], clean[p.starts[s]:at[s], 10:15])
        assert not torch.isfinite(out[at[s]:p.starts[s] + n, 10:15, 5]).any()
        held = c.vc[s, 2, b + at[s] - p.starts[s], 5].item()
        assert math.isnan(held) if math.isnan(what) else held == what
