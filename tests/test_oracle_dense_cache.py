"""Pins of the bounded dense caches' plain reference (oracle/dense_cache.py):
the attention against a library softmax, the weights against its column sums,
and the choice of what stays against worked cases."""
import numpy as np
import pytest

from oracle import dense_cache as dc


@pytest.mark.parametrize("before,n", [(0, 7), (5, 1), (9, 4)])
def test_attend_against_a_library_softmax(before, n):
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(before + n)
    Hq, Hkv, L = 6, 2, before + n
    q, k, v = rng.normal(size=(n, Hq, dc.D)), rng.normal(size=(Hkv, L, dc.D)), rng.normal(size=(Hkv, L, dc.D))
    out, lse, mag, size = dc.attend(q, k, v, 0.1, before)
    kk, vv = (torch.from_numpy(x).repeat_interleave(3, 0) for x in (k, v))
    a = torch.einsum("nhd,hld->hnl", torch.from_numpy(q), kk) * 0.1
    a = a.masked_fill(torch.arange(L) > before + torch.arange(n)[:, None], -np.inf)
    w = torch.softmax(a, -1)
    np.testing.assert_allclose(out, torch.einsum("hnl,hld->nhd", w, vv).numpy(), atol=1e-13)
    np.testing.assert_allclose(lse, torch.logsumexp(a, -1).T.numpy(), atol=1e-13)
    assert np.all(np.abs(out) <= mag + 1e-13)
    assert np.all(np.abs(np.where(np.isinf(a), 0, a.numpy())).max(-1).T <= size + 1e-13)
    for window in (0, 1, n, n + 3):
        first = max(0, n - window)
        want = w[:, first:].sum(1).view(Hkv, 3, L).sum(1).numpy()
        np.testing.assert_allclose(dc.received(q, k, 0.1, before, lse, window), want, atol=1e-13)


def test_what_stays():
    assert dc.kept([3.0, 1.0, 2.0], 3, 0) == [0, 1, 2] and dc.kept([], 2, 1) == []
    assert dc.kept([3.0, 1.0, 2.0], 2, 0) == [0, 2]
    assert dc.kept([3.0, 1.0, 2.0], 2, 1) == [0, 2] and dc.kept([3.0, 1.0, 2.0], 2, 2) == [1, 2]
    assert dc.kept([1.0, 1.0, 1.0, 1.0], 2, 0) == [0, 1] and dc.kept([1.0, 1.0, 2.0, 0.0], 3, 1) == [0, 2, 3]
    assert dc.kept([0.0, -0.0, 0.0, -1.0], 2, 0) == [0, 1]
    assert dc.kept([np.inf, 1.0, np.nan, 5.0], 1, 0) == [2] and dc.kept([np.inf, 1.0, np.nan, 5.0], 2, 0) == [0, 2]
