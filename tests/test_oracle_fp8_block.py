"""Pins of the fp64 oracle of FP8 blocks of 128 and of the norm (CPU)."""
import numpy as np
import torch

from oracle import fp8_block as fb, mx


def test_quantize_by_hand():
    x = np.zeros((2, 160), np.float32)
    x[0, :4] = [448, 1, -0.0625, 17]      # scale 1: E4M3 rounds 17 (spacing 2) to the even code, 16
    x[1, 128] = 7                          # second block: scale 7 / 448
    q, s = fb.quantize(x)
    assert s.shape == (2, 2) and s[0, 0] == 1 and s[1, 1] == np.float32(7) / np.float32(448)
    assert s[0, 1] == np.float32(2.0 ** -100) / np.float32(448)
    v = fb.decode(q, s)
    assert list(v[0, :4]) == [448, 1, -0.0625, 16] and abs(v[1, 128] - 7) <= 7 * 2.0 ** -24
    assert not v[0, 4:].any()


def test_codes_are_torchs():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((40, 300)) * np.exp2(rng.integers(-8, 8, (40, 1)))).astype(np.float32)
    q, s = fb.quantize(x)
    for b in range(3):
        k = slice(128 * b, min(300, 128 * b + 128))
        m = np.abs(x[:, k]).max(1)
        t = torch.from_numpy(x[:, k] * (np.float32(448) / m)[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        np.testing.assert_array_equal(q[:, k], t.view(torch.uint8).numpy())
        np.testing.assert_array_equal(s[:, b], m / np.float32(448))


def test_error_is_half_a_step():
    """A value is off by at most half a step: 2^-4 of itself, or half of E4M3's smallest step (2^-10) times the scale."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((260, 290))
    for tile in (False, True):
        q, s = fb.quantize(x, tile)
        v = fb.decode(q, s, tile)
        assert np.all(np.abs(v - x) <= np.maximum(np.abs(x) * 2.0 ** -4, fb.spread(s, 260, 290, tile) * 2.0 ** -10) * (1 + 1e-6))


def test_tile_and_transpose():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((200, 330)).astype(np.float32)
    q, s = fb.quantize(x, True)
    qc, sc = fb.quantize_cols(x, True)
    assert s.shape == (2, 3)
    np.testing.assert_array_equal(sc, s.T)
    np.testing.assert_array_equal(qc[:, :200], q.T)
    assert qc.shape == (330, 224) and not qc[:, 200:].any()


def test_bad_block():
    x = np.ones((2, 200), np.float32)
    x[0, 3], x[1, 150] = np.inf, np.nan
    _, s = fb.quantize(x)
    np.testing.assert_array_equal(np.isnan(s), [[True, False], [False, True]])


def test_rmsnorm_gradients_by_differences():
    rng = np.random.default_rng(3)
    r, w, dy = rng.standard_normal((3, 32)), rng.standard_normal(32), rng.standard_normal((3, 32))
    _, rstd = fb.rmsnorm(r, w, 1e-2)
    dx, dw = fb.rmsnorm_bwd(dy, r, w, rstd)
    h = 1e-6
    for i in range(3):
        for j in range(0, 32, 7):
            p, q = r.copy(), r.copy()
            p[i, j] += h
            q[i, j] -= h
            d = ((fb.rmsnorm(p, w, 1e-2)[0] - fb.rmsnorm(q, w, 1e-2)[0]) * dy).sum() / (2 * h)
            assert abs(d - dx[i, j]) < 1e-6
    for j in range(32):
        p, q = w.copy(), w.copy()
        p[j] += h
        q[j] -= h
        d = ((fb.rmsnorm(r, p, 1e-2)[0] - fb.rmsnorm(r, q, 1e-2)[0]) * dy).sum() / (2 * h)
        assert abs(d - dw[j]) < 1e-6
    assert mx.e4m3_decode(np.array([0x7E], np.uint8))[0] == 448
