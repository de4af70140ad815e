"""Pins of the oracle's norm and rotation and of its 4-bit rows: closed forms,
complex arithmetic and round trips."""
import numpy as np
import pytest

import oracle as O


def test_norm_is_the_unit_root_mean_square():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 2, 64)) * 7
    y = O.norm_rope(x, None, 0.0, np.zeros(3), np.zeros(4), -1, True)
    assert np.allclose((y ** 2).mean(axis=-1), 1.0, rtol=1e-14)
    assert np.allclose(y * np.sqrt((x ** 2).mean(axis=-1, keepdims=True)), x, rtol=1e-13)
    w = rng.standard_normal(64)
    assert np.allclose(O.norm_rope(x, w, 0.0, None, [], -1, True), y * w, rtol=1e-14)
    # a huge eps leaves x / sqrt(eps)
    assert np.allclose(O.norm_rope(x, None, 1e12, None, [], -1, True), x / 1e6, rtol=1e-9)


@pytest.mark.parametrize("interleaved", [True, False])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 3, 24))
    pos = np.array([0, 1, 7, 1000, 99999])
    f = np.array([1.0, 0.3, 0.01, 1e-4])
    y = O.norm_rope(x, None, 0.0, pos, f, 8, interleaved, scale=1.5, norm=False)
    r = x[..., 8:16]
    z = r[..., 0::2] + 1j * r[..., 1::2] if interleaved else r[..., :4] + 1j * r[..., 4:]
    z = 1.5 * z * np.exp(1j * pos[:, None, None] * f)
    got = y[..., 8:16]
    got = got[..., 0::2] + 1j * got[..., 1::2] if interleaved else got[..., :4] + 1j * got[..., 4:]
    assert np.allclose(got, z, rtol=1e-12)
    assert np.array_equal(y[..., :8], x[..., :8]) and np.array_equal(y[..., 16:], x[..., 16:])
    assert np.array_equal(y[0], np.concatenate([x[0, :, :8], 1.5 * x[0, :, 8:16], x[0, :, 16:]], -1))


def test_rotated_products_depend_on_the_distance_alone():
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((2, 1, 1, 16))
    f = 100.0 ** -np.linspace(0, 1, 8, endpoint=False)

    def dot(i, j):
        a = O.norm_rope(q, None, 0.0, [i], f, 0, True, norm=False)
        b = O.norm_rope(k, None, 0.0, [j], f, 0, True, norm=False)
        return float((a * b).sum())
    assert abs(dot(10, 3) - dot(107, 100)) < 1e-12
    assert abs(dot(10, 3) - dot(10, 4)) > 1e-3


def test_4_bit_rows():
    rng = np.random.default_rng(3)
    v = (rng.standard_normal((6, 512)) * np.exp(rng.standard_normal((6, 1)) * 4)).astype(np.float32)
    v[2, :32] = 0
    rows = O.latent_rows_mxfp4(v)
    assert rows.shape == (6, 272) and rows.dtype == np.uint8
    back = O.latent_values(rows, "mxfp4")
    # a row's values come back as themselves, and are theirs to within half a step
    assert np.array_equal(O.latent_values(O.latent_rows_mxfp4(back.astype(np.float32)), "mxfp4"), back)
    amax = np.abs(v.reshape(6, 16, 32)).max(axis=-1)
    err = np.abs(back - v).reshape(6, 16, 32).max(axis=-1)
    assert np.all(err <= amax / 4 + 1e-30)  # at most 2 of 8 at the group's top (6 from 8 - 0)
    assert rows[2, 256] == 127 and not rows[2, :16].any()
    # element 2 i in the low nibble of byte i; scale g of elements 32 g ..
    one = np.zeros((1, 512), np.float32)
    one[0, 33] = -3.0
    r = O.latent_rows_mxfp4(one)[0]
    assert O.latent_values(r, "mxfp4")[33] == -3.0 and np.count_nonzero(r[:256]) == 1
    assert r[16] & 0x0F == 0 and r[16] >> 4 >= 8
    assert r[256 + 1] == 127 + 1 - 2 and r[256] == 127
