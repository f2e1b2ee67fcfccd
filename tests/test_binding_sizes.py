"""Sizes past 31 bits in the Python calls of the norm and of FP8 with scales for blocks of 128 (CPU, tensors without
memory): the argument blocks hold them in 32 bits, so a call on such a tensor is refused before it would be made for
the size's low bits."""
import pytest
import torch

from moe_grouped_expert_amd import _binding as b

BIG = (1 << 32) + 32      # low 32 bits: 32, a size that every call takes


@pytest.fixture(autouse=True)
def no_gpu(monkeypatch):
    monkeypatch.setattr(b, "_on", lambda dev, *ts: None)

    def call(fn, a, dev):
        pytest.fail(f"{fn} was called with " + ", ".join(f"{n}={getattr(a, n)}" for n, t in a._fields_ if t is b.i32))

    monkeypatch.setattr(b, "_call", call)


def empty(shape, dt=torch.bfloat16):
    return torch.empty(shape, dtype=dt, device="meta")


U8, F32, I32 = torch.uint8, torch.float32, torch.int32
NB = (BIG + 127) // 128


def operand(rows, K):
    return empty((rows, K), U8), empty((rows, (K + 127) // 128), F32)


CALLS = {
    "rmsnorm_fwd columns": lambda: b.rmsnorm_fwd(empty((1, BIG)), empty((BIG,))),
    "rmsnorm_fwd rows": lambda: b.rmsnorm_fwd(empty((BIG, 32)), empty((32,))),
    "rmsnorm_fwd leading sizes": lambda: b.rmsnorm_fwd(empty((1 << 16, 1 << 16, 32)), empty((32,))),
    "rmsnorm_fwd strided rows": lambda: b.rmsnorm_fwd(empty((BIG, 64))[:, :32], empty((32,))),
    "rmsnorm_bwd rows": lambda: b.rmsnorm_bwd(empty((BIG, 32)), empty((BIG, 32)), empty((32,)), empty((BIG,), F32), want_dw=False),
    "rmsnorm_bwd columns": lambda: b.rmsnorm_bwd(empty((1, BIG)), empty((1, BIG)), empty((BIG,)), empty((1,), F32), want_dw=False),
    "quantize columns": lambda: b.fp8_block_quantize(empty((1, BIG))),
    "quantize rows": lambda: b.fp8_block_quantize(empty((BIG, 32))),
    "quantize batch": lambda: b.fp8_block_quantize(empty((BIG, 1, 32))),
    "quantize mapped rows": lambda: b.fp8_block_quantize(empty((32, 32)), rows=empty((BIG,), I32)),
    "dequantize columns": lambda: b.fp8_block_dequantize(empty((1, BIG), U8), empty((1, NB), F32)),
    "dequantize rows": lambda: b.fp8_block_dequantize(empty((BIG, 32), U8), empty((BIG, 1), F32)),
    "dequantize batch": lambda: b.fp8_block_dequantize(empty((BIG, 1, 32), U8), empty((BIG, 1, 1), F32)),
    "gemm K": lambda: b.fp8_block_grouped_gemm(*operand(1, BIG), empty((1, 32, BIG), U8), empty((1, 1, NB), F32)),
    "gemm N": lambda: b.fp8_block_grouped_gemm(*operand(1, 32), empty((1, BIG, 32), U8), empty((1, NB, 1), F32)),
    "wgrad N": lambda: b.fp8_block_grouped_wgrad(*operand(BIG, 32), *operand(32, 32)),
    "wgrad K": lambda: b.fp8_block_grouped_wgrad(*operand(32, 32), *operand(BIG, 32)),
    "mlp H": lambda: b.grouped_mlp_fwd_fp8_block(None, *operand(1, BIG), empty((1, 64, BIG), U8), empty((1, BIG, 32), U8),
                                                 empty((1, 1, NB), F32), empty((1, NB, 1), F32)),
    "mlp F": lambda: b.grouped_mlp_fwd_fp8_block(None, *operand(1, 32), empty((1, 2 * BIG, 32), U8), empty((1, 32, BIG), U8),
                                                 empty((1, 2 * NB, 1), F32), empty((1, 1, NB), F32)),
}


@pytest.mark.parametrize("name", CALLS)
def test_sizes_past_31_bits_are_refused(name):
    with pytest.raises(ValueError, match="2\\^31"):
        CALLS[name]()


def test_smaller_sizes_reach_the_library(monkeypatch):
    """... as they are."""
    seen = []
    monkeypatch.setattr(b, "_call", lambda fn, a, dev: seen.append((fn, a)))
    H = (1 << 31) - 32
    b.rmsnorm_fwd(empty((1, H)), empty((H,)))
    b.fp8_block_quantize(empty((3, H)))
    assert [(fn, a.T, a.H) if fn == "rmsnorm_fwd" else (fn, a.R, a.C) for fn, a in seen] == [("rmsnorm_fwd", 1, H), ("fp8_block_quantize", 3, H)]
