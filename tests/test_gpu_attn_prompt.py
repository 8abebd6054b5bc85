"""GPU parity of the attention of packed whole prompts over the dense caches
(mamba2_attn_prompt) against its plain reference (oracle/dense_cache.py),
through the C ABI. The bounds stand in tests/dense_cache_lib.py."""
import math

import numpy as np
import pytest

from dense_cache_lib import D, Caches, Packed, dtype

pytestmark = pytest.mark.gpu

HEADS = [(40, 8), (4, 4), (8, 1), (14, 2), (12, 2), (9, 3), (6, 3), (4, 1)]


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


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_head_layouts(m2, act, Hq, Hkv):
    """1 to 8 query heads a kv head; an empty cache, one in use, a session without new rows."""
    c = Caches(m2, [0, 37, 130, 5], Hq, Hkv, act, 300, seed=Hq)
    p = Packed(c, [70, 1, 61, 0], lead=2, tail=3, pad=8)
    p.attend()
    _done(m2)
    p.check()


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("before,new", [
    ([0], [1]), ([0], [2]), ([0], [25]), ([0], [26]), ([0], [50]), ([0], [51]), ([0], [300]),
    ([63, 64, 65, 127, 128, 129], [1, 1, 1, 1, 1, 1]),
    ([127, 126, 128, 255, 256, 200], [2, 2, 1, 3, 129, 57]),
    ([0, 0, 0], [128, 127, 129]),
    ([640], [1]), ([1000], [33]),
])
def test_lengths(m2, act, before, new):
    """One token to some hundred, around the tiles' and chunks' edges, up to the cache's last slot."""
    c = Caches(m2, before, 10, 2, act, max(b + n for b, n in zip(before, new)), seed=sum(new))
    p = Packed(c, new)
    p.attend()
    _done(m2)
    p.check()


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_many_short_sessions(m2, act):
    """More sessions than a block has threads, of no row to three."""
    rng = np.random.default_rng(5)
    new = rng.integers(0, 4, 700).tolist()
    c = Caches(m2, rng.integers(0, 20, 700).tolist(), 5, 1, act, 24, seed=1)
    p = Packed(c, new, lead=1, tail=1)
    p.attend()
    _done(m2)
    p.check()


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_no_lengths_means_empty_caches(m2, act):
    c = Caches(m2, [0, 0], 8, 2, act, 90, seed=2)
    p = Packed(c, [90, 41])
    p.attend(lengths=None, lse=False)
    _done(m2)
    p.check(lse=False)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [0.0, -0.05, 3.0])
def test_scales(m2, act, scale):
    c = Caches(m2, [20, 0], 8, 2, act, 200, seed=3, spread=0.5)
    p = Packed(c, [150, 60])
    p.attend(scale=scale)
    _done(m2)
    p.check()


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_large_and_tiny_scores(m2, act):
    """Scores of thousands, whose maximum moves along the row, and of 1e-30."""
    c = Caches(m2, [0], 5, 1, act, 400, seed=4)
    p = Packed(c, [400])
    p.q.mul_(40.0)
    p.attend()
    _done(m2)
    p.check()
    p.q.mul_(1e-32)
    p.attend()
    _done(m2)
    p.check()


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("at,what", [(0, math.inf), (3, math.nan), (31, math.nan), (60, -math.inf), (149, math.nan)])
def test_values_that_are_not_finite_reach_the_rows_that_see_them(m2, act, at, what):
    import torch
    before = 20
    c = Caches(m2, [before, 40], 10, 2, act, 200, seed=6)
    p = Packed(c, [150, 30])
    clean = Packed(Caches(m2, [before, 40], 10, 2, act, 200, seed=6), [150, 30])
    clean.attend()
    p.v[at, 7] = what  # one dim of kv head 0
    p.attend()
    _done(m2)
    sees = torch.arange(150, device="cuda") >= at
    heads = p.out[:150].view(150, 10, D).float()
    assert torch.all(~torch.isfinite(heads[sees][:, :5, 7]))
    assert torch.equal(heads[~sees], clean.out[:150].view(150, 10, D).float()[~sees])
    assert torch.equal(heads[:, 5:], clean.out[:150].view(150, 10, D).float()[:, 5:])
    assert torch.equal(p.out[150:], clean.out[150:]) and torch.equal(p.lse, clean.lse)


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_keys_and_queries_that_are_not_finite(m2, act):
    """A key reaches the rows that see it, a query its own row and head."""
    import torch
    c = Caches(m2, [0], 4, 2, act, 160, seed=7)
    p = Packed(c, [160])
    clean = Packed(Caches(m2, [0], 4, 2, act, 160, seed=7), [160])
    clean.attend()
    p.k[100, 3] = math.nan        # kv head 0
    p.q[20, 3 * D + 1] = math.inf  # head 3
    p.attend()
    _done(m2)
    out, want = p.out.view(160, 4, D).float(), clean.out.view(160, 4, D).float()
    assert torch.isnan(out[100:, :2]).all() and torch.equal(out[:100, :2], want[:100, :2])
    assert not torch.isfinite(out[20, 3]).any() and torch.equal(out[20, 2], want[20, 2])
    assert torch.equal(out[21:, 2:], want[21:, 2:]) and torch.equal(out[:20, 2:], want[:20, 2:])


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_refused_sessions(m2, act):
    """Lengths that the host does not see: zeros, -infinity, untouched caches; the others as usual."""
    import torch
    c = Caches(m2, [10, 91, -3, 60], 10, 2, act, 100, seed=8)
    p = Packed(c, [30, 10, 4, 40])
    held = c.kc.clone(), c.vc.clone()
    p.attend()
    _done(m2, 0x104)
    p.check(sessions=[0, 3])
    for s in (1, 2):
        assert torch.all(p.out[p.mine(s)] == 0) and torch.all(p.lse[p.mine(s)] == -math.inf)
        for now, old in zip((c.kc, c.vc), held):
            assert torch.equal(now[s].view(torch.uint8), old[s].view(torch.uint8))


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("starts", [[0, 30, 99], [-4, 30, 70], [0, 40, 30], [75, 75, 2000000000]])
def test_row_starts_outside_the_rows_are_recorded(m2, act, starts):
    """A session whose rows do not lie within the call's is left out."""
    import torch
    c = Caches(m2, [0, 5], 10, 2, act, 100, seed=9)
    p = Packed(c, [30, 40])
    held = c.kc.clone()
    p.attend(row_start=torch.tensor(starts, dtype=torch.int32, device="cuda"))
    _done(m2, 0x106)
    for s in range(2):
        if not 0 <= starts[s] <= starts[s + 1] <= 70:
            assert torch.equal(c.kc[s].view(torch.uint8), held[s].view(torch.uint8))
    good = Packed(Caches(m2, [0, 5], 10, 2, act, 100, seed=9), [30, 40])
    good.attend()
    _done(m2)
    good.check()


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_split_anywhere_gives_the_same_attention(m2, act):
    """A prompt in one call or in several, one token at the end: the same caches, outputs within the bounds."""
    import torch
    c = Caches(m2, [0], 10, 2, act, 150, seed=10)
    p = Packed(c, [150])
    p.attend()
    _done(m2)
    p.check()
    d = Caches(m2, [0], 10, 2, act, 150, seed=11)
    at = 0
    for n in (64, 1, 60, 24, 1):
        d.before, d.lengths = [at], torch.tensor([at], dtype=torch.int32, device="cuda")
        q = Packed(d, [n])
        q.rows[:] = p.rows[at:at + n]
        q.attend()
        _done(m2)
        q.check()
        at += n
    assert torch.equal(c.kc, d.kc) and torch.equal(c.vc, d.vc)


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_another_stream_and_a_replayed_graph(m2, act):
    import torch
    c = Caches(m2, [30, 0], 10, 2, act, 200, seed=12)
    p = Packed(c, [100, 77])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    p.attend(stream=side)
    _done(m2)
    p.check()
    want = p.out.clone(), p.lse.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.attend()
    for _ in range(2):
        p.out.fill_(-7.0), p.lse.fill_(-7.0)
        c.kc[0, :, 30:130] = math.nan
        graph.replay()
        _done(m2)
        assert torch.equal(p.out, want[0]) and torch.equal(p.lse, want[1])
    p.check()


def test_offsets_past_32_bits(m2):
    """Caches of more than 2^31 elements, the last session at the end of its slots."""
    import torch
    S, Hkv, max_len = 36, 8, 60000
    assert S * Hkv * max_len * D > 2 ** 31
    c = Caches.__new__(Caches)
    c.m2, c.Hq, c.Hkv, c.act, c.max_len, c.S, c.spread = m2, 40, Hkv, "bf16", max_len, S, 1.0
    c.g = torch.Generator().manual_seed(13)
    c.kc, c.vc = (torch.zeros(S, Hkv, max_len, D, dtype=dtype("bf16"), device="cuda") for _ in "kv")
    c.before = [0] * (S - 1) + [max_len - 60]
    c.lengths = torch.tensor(c.before, dtype=torch.int32, device="cuda")
    p = Packed(c, [0] * (S - 2) + [9, 60])
    p.attend()
    _done(m2)
    s = S - 1
    want = p.k[9:69, :Hkv * D].reshape(60, Hkv, D).transpose(0, 1)
    assert torch.equal(c.kc[s, :, max_len - 60:], want)
    # keys and values before are zeros: a row's weights are those of its own, and of so many zeros
    q, k, v = (x[9:69].double().cpu() for x in (p.q[:, :40 * D], p.k[:, :Hkv * D], p.v[:, :Hkv * D]))
    for t in (0, 59):
        for h in (0, 39):
            a = (k[:t + 1].view(-1, Hkv, D)[:, h // 5] @ q[t].view(40, D)[h]) * D ** -0.5
            w = torch.exp(a)
            total = w.sum() + (max_len - 60)
            assert abs(p.lse[9 + t, h].item() - math.log(total)) < 1e-4
            want = (w[:, None] * v[:t + 1].view(-1, Hkv, D)[:, h // 5]).sum(0) / total
            got = p.out[9 + t].view(40, D)[h].double().cpu()
            # a weight may be rounded to 2^-8 of itself, and 1e-4 for fp32 scores and sums
            mag = (w[:, None] * v[:t + 1].view(-1, Hkv, D)[:, h // 5].abs()).sum(0) / total
            assert torch.all((got - want).abs() <= (2 ** -8 + 1e-4) * mag + 2 ** -8 * want.abs())


@pytest.mark.parametrize("before", [0, 1, 127, 128, 129, 255, 256])
@pytest.mark.parametrize("new", [1, 49, 50, 51, 127, 128, 129, 257])
def test_appended_whatever_lies_around(m2, before, new):
    """Every new row in the caches bit for bit, NaN and infinities among them, and no slot more: one to three
    sessions, whose rows' chunks begin anywhere in a tile."""
    import torch
    c = Caches(m2, [before, 3, before], 10, 2, "bf16", before + new + 5, seed=70)
    p = Packed(c, [new, 2, max(0, new - 40)], lead=1, tail=1)
    p.k[2, 5], p.v[1 + new // 2, 200], p.v[new, 3] = math.nan, math.inf, -math.inf
    p.attend()
    _done(m2)
    for s in range(3):
        b, n = c.before[s], p.new[s]
        for cache, rows in ((c.kc, p.k), (c.vc, p.v)):
            want = rows[p.mine(s), :2 * D].reshape(n, 2, D).transpose(0, 1).contiguous()
            assert torch.equal(cache[s, :, b:b + n].contiguous().view(torch.uint8), want.view(torch.uint8))
            assert torch.isnan(cache[s, :, b + n:]).all()
