"""How large and how small the scales of FP8 blocks may be in the products and the weight gradient: inside the documented
range sums of equal powers of two are exact (every partial sum is a small integer times one power of two, so there is no
rounding to allow for); past it only the elements whose blocks they are lose their values."""
import numpy as np
import pytest
import torch

from oracle import mx
from tests.test_gpu_fp8_block import gpu, groups, m, npy  # noqa: F401

pytestmark = pytest.mark.gpu

# rows, N, K: streamed, quadrants alone, whole tiles and quadrants
FORMS = [(5, 160, 544), (200, 288, 544), (4100, 2080, 288)]


def codes(rng, shape, top):
    """Integers up to `top` and their codes."""
    v = rng.integers(-top, top + 1, shape).astype(np.float64)
    return v, mx.e4m3_encode(v)


def say(*a):
    from tests.gpu_helpers import say as s
    s("[gpu] range", *a)


@pytest.mark.parametrize("rows,N,K", FORMS)
@pytest.mark.parametrize("both", [127, 126, 0, -126, -140, -149])
def test_product_of_scales(m, rows, N, K, both):  # noqa: F811
    """a_scale w_scale = 2^both, split between the two in every way the rows and blocks offer."""
    say("product", rows, N, K, both)
    rng = np.random.default_rng(rows + both + 200)
    nb, nn = (K + 127) // 128, (N + 127) // 128
    # 2^both times the sums has to be finite: at the top codes of +-2^-9, E4M3's smallest
    unit = 2.0 ** -9 if both > 100 else 1.0
    a, w = rng.integers(-1, 2, (rows, K)).astype(np.float64), rng.integers(-1, 2, (N, K)).astype(np.float64)
    ea = np.broadcast_to(rng.integers(max(-100, both - 100), min(101, both + 101), nb), (rows, nb))
    ew = np.broadcast_to(both - ea[:1], (nn, nb))
    got = m.fp8_block_grouped_gemm(gpu(mx.e4m3_encode(a * unit)), gpu(np.exp2(ea.astype(np.float64)), np.float32), gpu(mx.e4m3_encode(w * unit))[None],
                                   gpu(np.exp2(ew.astype(np.float64)), np.float32)[None], out_dtype="f32")
    np.testing.assert_array_equal(npy(got).astype(np.float64), np.ldexp((a @ w.T) * unit * unit, both))


@pytest.mark.parametrize("rows,N,K", FORMS)
def test_product_past_the_range_stays_in_its_elements(m, rows, N, K):  # noqa: F811
    say("past", rows, N, K)
    rng = np.random.default_rng(rows)
    nb, nn = (K + 127) // 128, (N + 127) // 128
    a, ac = codes(rng, (rows, K), 3)
    w, wc = codes(rng, (N, K), 3)
    a_s, w_s = np.ones((rows, nb), np.float32), np.ones((nn, nb), np.float32)
    ref = a @ w.T
    a_s[3, 1] = 2.0 ** 100
    w_s[1, 1] = 2.0 ** 100
    got = npy(m.fp8_block_grouped_gemm(gpu(ac), gpu(a_s), gpu(wc)[None], gpu(w_s)[None], out_dtype="f32")).astype(np.float64)
    plain = np.ones((rows, N), bool)
    plain[:, 128:256] = False     # one large scale or two
    plain[3] = False
    np.testing.assert_array_equal(got[plain], ref[plain])
    assert not np.isfinite(got[3, 128:256]).any()
    got[3, 128:256] = 0
    assert np.isfinite(got).all()


@pytest.mark.parametrize("sizes,N,K", [([200, 0, 33], 288, 160), ([2500, 700, 0, 2600], 1312, 2080)])   # tiles of 128, of 256
@pytest.mark.parametrize("first,second", [(103, -100), (103, 0), (-100, -20), (-100, 110), (0, 103)])
def test_weight_gradient(m, sizes, N, K, first, second):  # noqa: F811
    """dy_scale up to 2^103, whatever x_scale is."""
    say("wgrad", len(sizes), N, K, first, second)
    rng = np.random.default_rng(N + first + 200)
    off, R = groups(sizes, 128)
    R = (R + 31) // 32 * 32
    inside = np.zeros(R, bool)
    for n, o in zip(sizes, off):
        inside[o:o + n] = True
    y, x = rng.integers(-1, 2, (N, R)).astype(np.float64) * inside, rng.integers(-1, 2, (K, R)).astype(np.float64) * inside
    nb = (R + 127) // 128
    got = m.fp8_block_grouped_wgrad(gpu(mx.e4m3_encode(y)), gpu(np.full((N, nb), 2.0 ** first), np.float32), gpu(mx.e4m3_encode(x)),
                                    gpu(np.full((K, nb), 2.0 ** second), np.float32), gpu(sizes, np.int32), gpu(off, np.int32))
    for e, (n, o) in enumerate(zip(sizes, off)):
        np.testing.assert_array_equal(npy(got[e]).astype(np.float64), np.ldexp(y[:, o:o + n] @ x[:, o:o + n].T, first + second))
