"""The forms of the FP8 block products that larger sizes select, with few rows of K and odd edges so that the fp64 oracle
stays quick: whole rounds of 256 x 256 tiles with and without quadrants behind them, SwiGLU in the product's epilogue, and
the weight gradient's tiles of 256 x 256."""
import pytest

from tests.test_gpu_fp8_block import m, run_gemm, run_mlp, run_wgrad  # noqa: F401

pytestmark = pytest.mark.gpu


# tiles: 11 x 33 (a round, 107 as quadrants), 11 x 38 (a round and 162 more, all whole tiles), 24 x 21 (a round and 248)
@pytest.mark.parametrize("sizes,N,K", [([700, 0, 1025, 3, 511], 8224, 160), ([700, 0, 1025, 3, 511], 9536, 96),
                                       ([256] * 20 + [1, 2, 3, 100], 5344, 288)])
@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
def test_gemm_rounds(m, sizes, N, K, out_dtype):  # noqa: F811
    run_gemm(m, sizes, N, K, out_dtype, ints=True)
    run_gemm(m, sizes, N, K, out_dtype, align=32, extra=40, seed=2, stacked=False)
    run_gemm(m, sizes, N, K, out_dtype, ints=True, align=8, extra=9, seed=3, gather=True)


def test_gemm_rounds_of_many_experts(m):  # noqa: F811
    run_gemm(m, [(e * 37) % 150 for e in range(70)], 1056, 224, ints=True, align=8)


@pytest.mark.parametrize("T,E,k,H,F", [(500, 4, 2, 96, 4128), (1500, 4, 2, 160, 1440), (3000, 66, 2, 64, 288)])
def test_mlp_swiglu_in_the_epilogue(m, T, E, k, H, F):  # noqa: F811
    run_mlp(m, T, E, k, H, F)
    run_mlp(m, T, E, k, H, F, "f32", seed=1)


@pytest.mark.parametrize("T", [700])
def test_dense_mlp_swiglu_in_the_epilogue(m, T):  # noqa: F811
    run_mlp(m, T, 1, 1, 96, 5600, dense=True)


# groups of many, two, one and no slices, in turn
@pytest.mark.parametrize("sizes,N,K", [([3000, 0, 2100, 130, 1], 1056, 2080), ([1, 1500, 0, 128, 3000, 129], 2080, 2080)])
@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
def test_wgrad_large_tiles(m, sizes, N, K, out_dtype):  # noqa: F811
    run_wgrad(m, sizes, N, K, out_dtype, ints=True)
    run_wgrad(m, sizes, N, K, out_dtype, extra=160, seed=1)


def test_wgrad_large_tiles_accumulate(m):  # noqa: F811
    run_wgrad(m, [3000, 0, 2100, 130, 1], 1056, 2080, ints=True, accumulate=True)
    run_wgrad(m, [2500, 700, 0, 2600], 1312, 2080, seed=2, accumulate=True)
