"""Pins of the paged cache's plain reference (oracle/kv_paged.py): the e4m3
codec against torch's conversion and exact arithmetic, the rotation, the
quantisation bound and the attention against a library softmax."""
import numpy as np
import pytest

from oracle import kv_paged as kv


def test_e4m3_codec_against_torch():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.normal(size=20000) * 10.0 ** rng.uniform(-4, 2.4, 20000), kv.E4M3[np.isfinite(kv.E4M3)],
                        (kv.E4M3[:126] + kv.E4M3[1:127]) / 2, -(kv.E4M3[:126] + kv.E4M3[1:127]) / 2]).astype(np.float32)
    x = np.clip(x, -448, 448)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    got = kv.to_e4m3(x)
    np.testing.assert_array_equal(got, want)
    every = np.arange(256, dtype=np.uint8)
    np.testing.assert_array_equal(kv.E4M3, torch.from_numpy(every).view(torch.float8_e4m3fn).double().numpy())
    assert kv.to_e4m3(np.float32(np.nan)) == 0x7F and kv.to_e4m3(np.float32(1e9)) == 0x7E


def test_quantised_values_are_within_half_a_step():
    rng = np.random.default_rng(2)
    rows = (rng.normal(size=(37, 3, kv.D)) * np.exp(rng.normal(size=(37, 1, 1)))).astype(np.float32)
    rows[16:32, 1] = 0.0
    codes, scales = kv.quantise(rows)
    assert scales.shape == (3, 3)
    value = kv.E4M3[codes] * np.repeat(scales.astype(np.float64), kv.BLOCK, 0)[:37, :, None]
    step = np.repeat(scales.astype(np.float64), kv.BLOCK, 0)[:37, :, None]
    # half a step of e4m3, 2^-4 of the value, or 2^-10 of the scale below the
    # normals; 2^-22: the fp32 rounding of the scale
    assert np.all(np.abs(value - rows) <= (2.0 ** -4 + 2.0 ** -22) * np.abs(rows) + 2.0 ** -10 * step)
    assert np.all(codes[16:32, 1] == 0) and np.all(scales[1, 1] == kv.TINY / np.float32(448))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [16, 64, 128])
def test_rotation_is_a_complex_product(rot, interleaved):
    rng = np.random.default_rng(3)
    n, h = 9, rot // 2
    ang = rng.uniform(-3, 3, (40, h))
    x = rng.normal(size=(n, 2, kv.D))
    places = np.arange(11, 11 + n)
    y = kv.rotate(x, places, np.cos(ang), np.sin(ang), rot, interleaved, np.float64)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, h), slice(h, rot))
    z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * ang[places])[:, None]
    np.testing.assert_allclose(y[..., a], z.real, atol=1e-14)
    np.testing.assert_allclose(y[..., b], z.imag, atol=1e-14)
    np.testing.assert_array_equal(y[..., rot:], x[..., rot:])


def test_attend_against_a_library_softmax():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(4)
    n, Hq, Hkv, L = 5, 6, 2, 33
    q, k, v = rng.normal(size=(n, Hq, kv.D)), rng.normal(size=(L, Hkv, kv.D)), rng.normal(size=(L, Hkv, kv.D))
    seen = np.array([0, 1, 7, 32, 33])
    out, size, _, _ = kv.attend(q, k, v, 0.1, seen)
    a = torch.einsum("nhd,lhd->nhl", torch.from_numpy(q), torch.from_numpy(k).repeat_interleave(3, 1)) * 0.1
    a = a.masked_fill(torch.arange(L)[None, None] >= torch.from_numpy(seen)[:, None, None], -np.inf)
    w = torch.nan_to_num(torch.softmax(a, -1))
    want = torch.einsum("nhl,lhd->nhd", w, torch.from_numpy(v).repeat_interleave(3, 1)).numpy()
    np.testing.assert_allclose(out, want, atol=1e-13)
    assert np.all(out[0] == 0) and np.all(np.abs(out) <= size + 1e-13)
