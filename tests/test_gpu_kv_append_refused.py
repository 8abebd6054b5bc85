"""Sessions that mamba2_kv_append refuses on the device are left as they were,
also where the tails out are not the tails; and the error word tells the first
of several conditions."""
import numpy as np
import pytest

from test_gpu_kv_paged import BLOCK, Cache, _expected_pool, _int, _rope, _rows, _same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m2():
    import full_duplex_speech_gb300 as m2
    m2.load()
    return m2


@pytest.mark.parametrize("why", ["lengths", "rotation"])
@pytest.mark.parametrize("act,T", [("bf16", 1), ("f32", 37)])
def test_a_refused_session_keeps_its_tail_when_the_tails_are_swapped(m2, act, T, why):
    """A call between two others whose positions do not fit the table (or the
    rotation's table), or whose lengths are negative: the caller swaps the tails
    after every call, and the next block is still quantised from the session's
    own rows."""
    S, Hkv, ps, L = 4, 2, 16, 21
    cache = Cache(m2, S, Hkv, ps, L + 2 * T, act, seed=3, in_place=False)
    (k, kh), (v, vh) = _rows(1, S, L + T, Hkv, act), _rows(2, S, L + T, Hkv, act)

    def swap():
        cache.kt, cache.kto, cache.vt, cache.vto = cache.kto, cache.kt, cache.vto, cache.vt
        cache.desc = m2.kv_cache(S, Hkv, ps, cache.n_pages, cache.columns, cache.d_table, cache.kp, cache.vp, cache.ks,
                                 cache.vs, cache.kt, cache.vt, cache.kto, cache.vto, act=act)

    cache.append(k[:, :L], v[:, :L])
    swap()
    junk, _ = _rows(4, S, T, Hkv, act)
    if why == "lengths":
        cache.append(junk, junk, lengths=_int([cache.columns * ps - T + 1, -1, 2 ** 31 - 1, -(2 ** 31)]))
    else:
        cache.append(junk, junk, None, _rope(m2, 64, L, False)[0], lengths=_int([L] * S))
    assert m2.mamba2_device_error() == 0x104
    swap()
    cache.append(k[:, L:], v[:, L:], lengths=_int([L] * S))
    assert m2.mamba2_device_error() == 0
    for a, b in zip(cache.host(), _expected_pool(cache, [(kh[s], vh[s]) for s in range(S)])):
        _same(a, b)
    left = (L + T) % BLOCK
    for tail, rows in ((cache.kto, kh), (cache.vto, vh)):
        _same(tail[:, :, :left].cpu().numpy(), np.ascontiguousarray(rows[:, L + T - left:].transpose(0, 2, 1, 3)))


def test_the_error_word_keeps_the_first_condition(m2):
    """A bad length and a bad page in either order, and in one call."""
    cache = Cache(m2, 2, 1, 16, 40, "bf16")
    k, _ = _rows(1, 2, 3, 1, "bf16")
    q, _ = _rows(2, 2, 3, 4, "bf16")
    cache.append(k, k)
    table = cache.d_table.clone()

    def bad_length():
        cache.attend(q, True, lengths=_int([0, -1]))

    def bad_page(call):
        cache.d_table[0, 0] = cache.n_pages
        call()
        cache.d_table.copy_(table)

    assert m2.mamba2_device_error() == 0
    for first, second, code in ((bad_length, lambda: bad_page(lambda: cache.attend(q)), 0x104),
                                (lambda: bad_page(lambda: cache.append(k, k)), bad_length, 0x105)):
        first()
        second()
        assert m2.mamba2_device_error() == code
        assert m2.mamba2_device_error() == 0
    bad_page(bad_length)
    assert m2.mamba2_device_error() in (0x104, 0x105)
    assert m2.mamba2_device_error() == 0
