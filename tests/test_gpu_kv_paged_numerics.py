"""Attention over the paged cache where its arithmetic is stretched, in the form
for a few rows and in the tiles: values near the type's largest, one dominant
position before a long flat rest, queries with one wide channel, scores of any
finite size. The caches are written directly,
as codes and scales, so that the exact outputs are known."""
import math

import pytest

from oracle import kv_paged as kv
from test_gpu_kv_paged import BLOCK, D, Cache, _int
from test_gpu_kv_paged_forms import plan

pytestmark = pytest.mark.gpu

# (query heads, kv heads, positions a call): the rows form for 8 and for 16 rows, the tiles
FORMS = {"rows8": (4, 1, 1), "rows16": (12, 1, 1), "tiles": (80, 8, 128)}
ONE = 0x38  # the code of 1


@pytest.fixture(scope="module")
def m2():
    import full_duplex_speech_gb300 as m2
    m2.load()
    return m2


def cache_of(m2, Hkv, n, ps=128):
    """A cache of one session with n positions, all keys zero, all values 1."""
    cache = Cache(m2, 1, Hkv, ps, n, "bf16")
    cache.kp.zero_(), cache.vp.fill_(ONE), cache.ks.fill_(1.0), cache.vs.fill_(1.0)
    return cache


def at(cache, p):
    """Where position p lies: page, slot, block."""
    return int(cache.table[0, p // cache.ps]), p % cache.ps, p % cache.ps // BLOCK


def across(m2, cache, form, q_row, scale, n):
    """The outputs of equal queries q_row [D] over the first n positions."""
    import torch
    Hq, Hkv, T = FORMS[form]
    assert plan(m2, cache, T, Hq)[0] == form.rstrip("186")
    q = q_row.to(torch.bfloat16).cuda().expand(1, T, Hq, D).contiguous()
    out = cache.attend(q, False, None, scale=scale, lengths=_int([n]))
    assert m2.mamba2_device_error() == 0
    assert bool((out == out[0, 0, 0]).all()), "equal rows, equal outputs"
    return out[0, 0, 0].double().cpu().numpy()


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("late", [0.0, 9.0])
def test_values_near_the_largest(m2, form, late):
    """Values of 1.6e38 in a block that comes late and scores e^late times the
    others, whose values are 1: the output is those values' share, and finite."""
    import torch
    Hkv, n = FORMS[form][1], 400
    cache = cache_of(m2, Hkv, n)
    first = 384  # a block of the fourth chunk of 128
    page, slot, block = at(cache, first)
    cache.kp[page, :, slot:slot + BLOCK] = ONE
    cache.vp[page, :, slot:slot + BLOCK] = 0x7C  # 384
    cache.vs[page, :, block] = 2.0 ** 118
    q = torch.zeros(D)
    q[0] = 1.0
    got = across(m2, cache, form, q, late, n)
    share = BLOCK * math.exp(late) / (BLOCK * math.exp(late) + n - BLOCK)
    want = share * 384 * 2.0 ** 118
    # the weights to fp16, the softmax factor (scores up to 9: 2^-24 of them and 2^-22 of exp2), the rounding to bf16
    tol = 2.0 ** -8 + 2.0 ** -11 + 1e-5
    assert (abs(got - want) <= tol * want).all(), (got[0], want)


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("log2_weight", [-20, -25, -30])
def test_one_dominant_position_before_a_long_flat_rest(m2, form, log2_weight):
    """2^20 positions of equal weight behind one that outweighs each of them by
    2^-log2_weight, with values 1 and zero, so that what is dropped shows."""
    import torch
    Hkv, n = FORMS[form][1], 1 << 20
    cache = cache_of(m2, Hkv, n)
    page, slot, block = at(cache, 0)
    cache.kp[page, :, slot] = ONE
    cache.vp[page, :, slot] = 0
    q = torch.zeros(D)
    q[0] = 1.0
    got = across(m2, cache, form, q, -log2_weight * math.log(2.0), n)
    rest = (n - 1) * 2.0 ** log2_weight
    # weights of a power of two are fp16 numbers, and their fp32 sums exact; but below 2^-24 they are lost
    # in the sum that holds the dominant one, a quarter of the softmax's at most
    lost = rest / 4 if log2_weight < -24 else 0.0
    want = rest / (1 + rest)
    assert (abs(got - want) <= (2.0 ** -8 + 2.0 ** -11 + 1e-5 + lost) * want).all(), (got[0], want)


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("wide", [1.0, 300.0, 5000.0, 1e4, 1e5, 3e6])
def test_queries_with_one_wide_channel(m2, form, wide):
    """One channel of the queries is much wider than the others, and the keys are
    zero there, so that the scores are the other channels'. These may be off by
    2^-21 of the widest and 2^-3 of themselves in the tiles, not at all where
    they are 2^-13 of it or more, and not at all in the rows form."""
    import torch
    Hkv, n, small = FORMS[form][1], 400, 1.296875
    cache = cache_of(m2, Hkv, n)
    for p in range(0, n, 2):  # every other position scores 2 and is worth 1, the rest 0 and 0
        page, slot, _ = at(cache, p)
        cache.kp[page, :, slot, 1:] = ONE
    for p in range(1, n, 2):
        page, slot, _ = at(cache, p)
        cache.vp[page, :, slot] = 0
    q = torch.full((D,), small)
    q[0] = wide
    widest = float(q.to(torch.bfloat16)[0])
    got = across(m2, cache, form, q, 2 / (127 * small), n)
    off = 0.0
    if form == "tiles" and small < 2.0 ** -13 * widest:
        off = 2 * min(2.0 ** -21 * widest / small, 2.0 ** -3)
    # a softmax share moves by a quarter of the score at most; scores are fp32 sums of 128 products
    want = 1 / (1 + math.exp(-2))
    tol = (2.0 ** -8 + 2.0 ** -11 + 1e-5) * want + (off + 128 * 2.0 ** -24 * 2) / 4
    assert (abs(got - want) <= tol).all(), (got[0], want, tol)


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("n", [40, 700])
@pytest.mark.parametrize("power", [-112, -100, 112])
def test_scores_of_any_finite_size(m2, form, n, power):
    """Every score is +-2^112 or so; half of the positions, worth 1, score alike,
    and the other half, worth 0, score twice as far below zero."""
    import torch
    cache = cache_of(m2, FORMS[form][1], n)
    for p in range(n):
        page, slot, block = at(cache, p)
        low = (p // BLOCK) % 2 == 0
        cache.kp[page, :, slot, 0] = ONE
        cache.ks[page, :, block] = 2.0 ** (abs(power) // 2) * (2.0 if low == (power < 0) else 1.0)
        cache.vp[page, :, slot] = 0 if low else ONE
    q = torch.zeros(D)
    q[0] = math.copysign(2.0 ** (abs(power) // 2), power)
    assert (across(m2, cache, form, q, 1.0, n) == 1.0).all()
