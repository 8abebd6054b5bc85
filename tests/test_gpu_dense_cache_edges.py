"""The bounded dense caches at the edges of what their header allows. The bounds
stand in tests/dense_cache_lib.py; where a test has one of its own, it is derived
beside it."""
import math

import pytest

from dense_cache_lib import Caches, Packed

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
