"""Refusals of the norm and of the calls on FP8 with one scale per block of 128 (CPU): bad arguments come back as the
documented code with a message, before any launch; the Python entry points check shapes, types and devices."""
import ctypes as C
import os

import pytest
import torch

from moe_grouped_expert_amd import _binding as b

pytestmark = pytest.mark.skipif(not os.path.exists(b.LIB_PATH), reason="libmge.so not built")
P = 1 << 20    # a plausible, never dereferenced device address


def call(fn, st, **kw):
    a = st()
    a.struct_size = C.sizeof(st)
    for k, v in kw.items():
        setattr(a, k, v)
    r = getattr(b.lib(), fn)(C.byref(a), None)
    return r, b.lib().mge_last_error().decode()


NORM = dict(T=4, H=64, x_dtype=0, weight_dtype=1, y_dtype=0, eps=1e-6, x_row_stride=64, x=P, residual=P, weight=P,
            residual_out=P, y=P, codes=P, scales=P, rstd=P)


@pytest.mark.parametrize("kw,word", [
    (dict(T=-1), "T"), (dict(H=0), "H"), (dict(H=48), "H"), (dict(H=16416), "H"), (dict(x_dtype=2), "dtype"),
    (dict(weight_dtype=-1), "dtype"), (dict(y_dtype=5), "dtype"), (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"),
    (dict(eps=float("inf")), "eps"), (dict(x_row_stride=56), "stride"), (dict(x_row_stride=68), "stride"),
    (dict(residual=None), "residual"), (dict(residual_out=None), "residual"), (dict(codes=None), "codes"),
    (dict(scales=None), "scales"), (dict(y=None, codes=None, scales=None), "no output"), (dict(x=None), "NULL"),
    (dict(weight=None), "NULL"), (dict(x=P + 8), "misaligned"), (dict(weight=P + 4), "misaligned"), (dict(y=P + 8), "misaligned"),
    (dict(residual=P + 2), "misaligned"), (dict(residual_out=P + 8), "misaligned"), (dict(codes=P + 4), "misaligned"),
    (dict(scales=P + 2), "misaligned"), (dict(rstd=P + 1), "misaligned"), (dict(struct_size=8), "struct_size")])
def test_rmsnorm_fwd(kw, word):
    r, err = call("rmsnorm_fwd", b.RmsnormArgs, **{**NORM, **kw})
    assert r == b.MGE_ERR_INVALID_ARG and word in err, err


BWD = dict(T=4, H=64, x_dtype=0, weight_dtype=0, dy_dtype=0, x_row_stride=64, dy_row_stride=64, dy=P, x=P, weight=P, rstd=P,
           d_residual=P, dx=P, d_weight=P, workspace=P, workspace_bytes=1 << 20)


@pytest.mark.parametrize("kw,word", [
    (dict(T=-1), "T"), (dict(H=33), "H"), (dict(dy_dtype=2), "dtype"), (dict(x_row_stride=63), "stride"),
    (dict(dy_row_stride=32), "stride"), (dict(dy_row_stride=66), "stride"), (dict(dy=None), "NULL"), (dict(x=None), "NULL"),
    (dict(rstd=None), "NULL"), (dict(dx=None), "NULL"), (dict(dx=P + 8), "NULL or misaligned"), (dict(dy=P + 2), "misaligned"),
    (dict(d_residual=P + 8), "misaligned"), (dict(d_weight=P + 4), "d_weight"), (dict(workspace=P + 8), "aligned")])
def test_rmsnorm_bwd(kw, word):
    r, err = call("rmsnorm_bwd", b.RmsnormBwdArgs, **{**BWD, **kw})
    assert r == b.MGE_ERR_INVALID_ARG and word in err, err


def test_rmsnorm_workspaces_and_empty():
    L = b.lib()
    assert call("rmsnorm_bwd", b.RmsnormBwdArgs, **{**BWD, "workspace": None})[0] == b.MGE_ERR_WORKSPACE
    assert call("rmsnorm_bwd", b.RmsnormBwdArgs, **{**BWD, "workspace_bytes": 255})[0] == b.MGE_ERR_WORKSPACE
    assert L.mge_rmsnorm_bwd_workspace_bytes(0, 64) == L.mge_rmsnorm_bwd_workspace_bytes(4, 1 << 20) == 0
    assert L.mge_rmsnorm_bwd_workspace_bytes(4, 64) >= 256
    none = dict(x=None, weight=None, y=None, residual=None, residual_out=None, codes=None, scales=None, rstd=None)
    assert call("rmsnorm_fwd", b.RmsnormArgs, **{**NORM, **none, "T": 0})[0] == b.MGE_OK
    assert call("rmsnorm_bwd", b.RmsnormBwdArgs, **{**BWD, "T": 0, "d_weight": None, "dy": None, "workspace": None})[0] == b.MGE_OK


QUANT = dict(block=0, batch=1, R=4, C=64, in_batch_stride=256, in_row_stride=64, in_=P, orient=3, row_codes=P, row_scales=P,
             col_codes=P, col_scales=P)


@pytest.mark.parametrize("kw,word", [
    (dict(block=2), "block"), (dict(C=48), "multiple of 32"), (dict(C=(1 << 24) + 32), "2^24"), (dict(R=-1), "negative"),
    (dict(R=0x7fffffff), "at most"), (dict(batch=-1), "negative"), (dict(orient=0), "orient"), (dict(orient=4), "orient"),
    (dict(in_=None), "in must"), (dict(in_=P + 8), "aligned"), (dict(in_row_stride=56), "in_row_stride"),
    (dict(in_row_stride=68), "in_row_stride"), (dict(batch=2, in_batch_stride=128), "in_batch_stride"),
    (dict(rows=P, batch=2, in_batch_stride=256), "map"), (dict(rows=P, block=1), "map"), (dict(rows=P, src_rows=-1), "map"),
    (dict(rows=P + 2, src_rows=4), "map"), (dict(row_codes=None), "row"), (dict(row_scales=None), "row"),
    (dict(row_codes=P + 4), "row"), (dict(col_codes=None), "column"), (dict(col_scales=P + 1), "column")])
def test_quantize(kw, word):
    r, err = call("fp8_block_quantize", b.QuantFbArgs, **{**QUANT, **kw})
    assert r == b.MGE_ERR_INVALID_ARG and word in err, err


@pytest.mark.parametrize("kw", [dict(C=33), dict(R=-1), dict(batch=-1), dict(out_dtype=2), dict(block=3), dict(codes=None),
                                dict(codes=P + 1), dict(scales=None), dict(scales=P + 2), dict(out=None), dict(out=P + 2),
                                dict(C=0x7fffffe0)])
def test_dequantize(kw):
    base = dict(block=0, batch=1, R=4, C=64, out_dtype=0, codes=P, scales=P, out=P)
    assert call("fp8_block_dequantize", b.DequantFbArgs, **{**base, **kw})[0] == b.MGE_ERR_INVALID_ARG


def pointers(kw, names):
    w, bad = (b.vp * 2)(P, P), (b.vp * 2)(P, None)
    out = {n: C.cast(w, b.vp) for n in names}
    out.update({k: (C.cast(bad, b.vp) if v == "bad" else v) for k, v in kw.items()})
    return out, (w, bad)


def gemm(**kw):
    base = dict(E=2, N=64, K=64, rows=8, src_rows=8, split_sizes=P, group_offsets=P, a=P, a_scale=P, out_dtype=0, out=P,
                workspace=P, workspace_bytes=1 << 30)
    p, keep = pointers(kw, ("w", "w_scale"))
    return call("fp8_block_grouped_gemm", b.GemmFbArgs, **{**base, **p})


@pytest.mark.parametrize("kw,word", [
    (dict(E=0), "E"), (dict(E=257), "E"), (dict(N=48), "N and K"), (dict(N=(1 << 22) + 32), "N and K"), (dict(K=0), "N and K"),
    (dict(K=80), "N and K"), (dict(K=(1 << 22) + 32), "N and K"), (dict(rows=-1), "rows"), (dict(rows=1 << 25, src_rows=1 << 25), "rows"), (dict(src_rows=1 << 25, a_rows=P), "rows"),
    (dict(src_rows=9), "row map"), (dict(src_rows=-1, a_rows=P), "rows"), (dict(total_rows=-1), "total_rows"),
    (dict(N=1 << 22, K=1 << 10), "2^31"), (dict(split_sizes=None), "go together"), (dict(group_offsets=None), "go together"),
    (dict(split_sizes=None, group_offsets=None), "go together"), (dict(out_dtype=3), "out_dtype"), (dict(w=None), "NULL"),
    (dict(w="bad"), "expert 1"), (dict(w_scale="bad"), "expert 1"), (dict(a=None), "NULL"), (dict(a=P + 4), "misaligned"),
    (dict(a_scale=None), "NULL"), (dict(a_scale=P + 2), "misaligned"), (dict(a_rows=P + 1), "misaligned"), (dict(out=P + 8), "misaligned")])
def test_grouped_gemm(kw, word):
    r, err = gemm(**kw)
    assert r == b.MGE_ERR_INVALID_ARG and word in err, err


def wgrad(**kw):
    base = dict(E=2, N=64, K=96, rows=256, split_sizes=P, group_offsets=P, dy=P, dy_scale=P, x=P, x_scale=P, out_dtype=1, accumulate=0,
                workspace=P, workspace_bytes=1 << 30)
    p, keep = pointers(kw, ("dw",))
    return call("fp8_block_grouped_wgrad", b.WgradFbArgs, **{**base, **p})


@pytest.mark.parametrize("kw,word", [
    (dict(E=0), "E"), (dict(N=40), "N and K"), (dict(K=-32), "N and K"), (dict(K=(1 << 22) + 32), "N and K"), (dict(rows=100), "rows"),
    (dict(rows=-32), "rows"), (dict(rows=1 << 25), "rows"), (dict(rows=1 << 23), "rows"), (dict(split_sizes=None), "go together"), (dict(out_dtype=2), "out_dtype"),
    (dict(out_dtype=0, accumulate=1), "accumulate"), (dict(dw=None), "dw"), (dict(dw="bad"), "dw[1]"), (dict(dy=None), "NULL"),
    (dict(dy=P + 8), "misaligned"), (dict(dy_scale=P + 2), "misaligned"), (dict(x=P + 4), "misaligned"), (dict(x_scale=None), "NULL"),
    (dict(workspace=P + 8), "aligned")])
def test_grouped_wgrad(kw, word):
    r, err = wgrad(**kw)
    assert r == b.MGE_ERR_INVALID_ARG and word in err, err


def mlp(**kw):
    base = dict(E=2, H=64, F=96, rows=96, x_rows=4, split_sizes=P, group_offsets=P, perm_src=P, prob_perm=P, x=P, x_scale=P,
                y_dtype=0, y_perm=P, workspace=P, workspace_bytes=1 << 30)
    p, keep = pointers(kw, ("w_gate_up", "w_gate_up_scale", "w_down", "w_down_scale"))
    return call("grouped_mlp_fwd_fp8_block", b.FwdFbArgs, **{**base, **p})


@pytest.mark.parametrize("kw,word", [
    (dict(E=0), "E"), (dict(H=40), "H and F"), (dict(F=0), "H and F"), (dict(H=32, F=(1 << 21) + 32), "H and F"), (dict(H=(1 << 22) + 32), "H and F"), (dict(rows=-1), "rows"),
    (dict(rows=1 << 25), "rows"), (dict(x_rows=1 << 25), "rows"), (dict(perm_src=None), "perm_src"), (dict(total_rows=-1), "total_rows"),
    (dict(H=1 << 15, F=1 << 15), "2^31"), (dict(group_offsets=None), "go together"), (dict(y_dtype=2), "y_dtype"),
    (dict(w_down=None), "NULL"), (dict(w_gate_up="bad"), "w_gate_up[1]"), (dict(w_down_scale="bad"), "w_down[1]"), (dict(x=None), "NULL"),
    (dict(x_scale=P + 2), "misaligned"), (dict(y_perm=P + 8), "misaligned"), (dict(prob_perm=P + 1), "misaligned"),
    (dict(workspace=P + 8), "aligned")])
def test_mlp(kw, word):
    r, err = mlp(**kw)
    assert r == b.MGE_ERR_INVALID_ARG and word in err, err


def test_workspaces_and_empty():
    assert gemm(N=8192, rows=2000, src_rows=2000, workspace=None)[0] == b.MGE_ERR_WORKSPACE
    assert gemm(rows=0, src_rows=0, workspace=None, a=None, a_scale=None, out=None)[0] == b.MGE_OK
    assert wgrad(workspace_bytes=64)[0] == b.MGE_ERR_WORKSPACE
    assert mlp(workspace=None)[0] == b.MGE_ERR_WORKSPACE
    assert mlp(rows=0, x_rows=0, workspace=None, x=None, x_scale=None, y_perm=None)[0] == b.MGE_OK
    L = b.lib()
    for q in ("mge_gemm_fb_workspace_bytes", "mge_wgrad_fb_workspace_bytes", "mge_fwd_fb_workspace_bytes"):
        assert getattr(L, q)(None) == 0
    assert call("fp8_block_quantize", b.QuantFbArgs, **{**QUANT, "R": 0, "in_": None})[0] == b.MGE_OK
    assert call("fp8_block_dequantize", b.DequantFbArgs, block=0, batch=1, R=0, C=64)[0] == b.MGE_OK
    # more experts than pointers travel with a launch: a table, whatever the rows
    w = (b.vp * 65)(*[P] * 65)
    a = b.GemmFbArgs(struct_size=C.sizeof(b.GemmFbArgs), E=65, N=64, K=64, w=C.cast(w, b.vp), w_scale=C.cast(w, b.vp))
    assert L.mge_gemm_fb_workspace_bytes(C.byref(a)) >= 2 * 65 * 8


def test_python_checks():
    """Wrong dtypes, shapes and devices are refused before anything is allocated on a GPU."""
    import moe_grouped_expert_amd as m
    f, bf = torch.zeros, torch.bfloat16
    u8 = dict(dtype=torch.uint8)
    i32 = dict(dtype=torch.int32)
    q, s = f(4, 64, **u8), f(4, 1)
    w, ws = f(2, 32, 64, **u8), f(2, 1, 1)
    for fn in (lambda: m.rmsnorm_fwd(f(4, 64), f(64)),                                   # not on a GPU
               lambda: m.rmsnorm_fwd(f(4, 64, dtype=torch.float16), f(64)),
               lambda: m.rmsnorm_fwd(f(64, 4).t(), f(64)),
               lambda: m.rmsnorm_fwd(f(4, 64), f(64), form="fp8"),
               lambda: m.rmsnorm_fwd(f(4, 64), f(64), y_dtype="f16"),
               lambda: m.rmsnorm_bwd(f(4, 64), f(4, 32), f(64), f(4)),
               lambda: m.fp8_block_quantize(f(4, 64)),
               lambda: m.fp8_block_quantize(f(4, 64, dtype=bf)),
               lambda: m.fp8_block_quantize(f(4, 64, dtype=bf), "rows"),
               lambda: m.fp8_block_quantize(f(4, 64, dtype=bf), "row", "64x64"),
               lambda: m.fp8_block_quantize(f(64, 4, dtype=bf).t()),
               lambda: m.fp8_block_quantize(f(2, 4, 64, dtype=bf), rows=f(4, **i32)),
               lambda: m.fp8_block_dequantize(q, f(4, 2)),
               lambda: m.fp8_block_dequantize(q, s, "f16"),
               lambda: m.fp8_block_dequantize(q, s),
               lambda: m.fp8_block_grouped_gemm(q, f(4, 2), w, ws),
               lambda: m.fp8_block_grouped_gemm(q, s, w, ws, out_dtype="f16"),
               lambda: m.fp8_block_grouped_gemm(q, s, w, ws),
               lambda: m.fp8_block_grouped_wgrad(q, s, f(8, 96, **u8), f(8, 1)),
               lambda: m.fp8_block_grouped_wgrad(q, s, q, s),
               lambda: m.grouped_mlp_fwd_fp8_block(None, q, s, w, w, ws, ws),
               lambda: m.grouped_mlp_fwd_fp8_block(None, q, s, w[:1], w[:1], ws[:1], ws[:1], y_dtype="f16")):
        with pytest.raises(ValueError):
            fn()
