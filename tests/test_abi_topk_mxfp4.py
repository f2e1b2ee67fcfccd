"""Refusals of the router-choice and MXFP4 calls (CPU): bad arguments come back as the documented
code with a message, before any launch; the Python entry points check shapes and types."""
import ctypes as C
import os

import pytest
import torch

from moe_grouped_expert_amd import _binding as b

pytestmark = pytest.mark.skipif(not os.path.exists(b.LIB_PATH), reason="libmge.so not built")
P = 1 << 20    # a plausible, never dereferenced device address


def call(fn, st, keep=(), **kw):
    a = st()
    a.struct_size = C.sizeof(st)
    for k, v in kw.items():
        setattr(a, k, v)
    r = getattr(b.lib(), fn)(C.byref(a), None)
    return r, b.lib().mge_last_error().decode()


TOPK = dict(T=4, E=16, k=2, score=1, num_groups=4, topk_groups=2, group_topn=2, scale=1.0, logits_dtype=1,
            logits_row_stride=16, logits=P, topk_idx=P, topk_prob=P)
BWD = dict(T=4, E=16, k=2, score=0, scale=1.0, logits_dtype=0, logits_row_stride=16, logits=P, topk_idx=P, d_prob=P, d_logits=P)


@pytest.mark.parametrize("kw,word", [
    (dict(T=-1), "T"), (dict(E=0), "E"), (dict(E=257), "E"), (dict(k=0), "k"), (dict(k=9), "k"), (dict(E=3, k=4), "k"),
    (dict(score=2), "score"), (dict(logits_dtype=2), "dtype"), (dict(scale=float("inf")), "scale"),
    (dict(scale=float("nan")), "scale"), (dict(logits_row_stride=15), "stride"), (dict(logits=None), "NULL"),
    (dict(logits=P + 2), "misaligned"), (dict(topk_idx=None), "NULL"), (dict(topk_prob=None), "NULL"),
    (dict(num_groups=3), "num_groups"), (dict(num_groups=0), "num_groups"), (dict(topk_groups=0), "topk_groups"),
    (dict(topk_groups=5), "topk_groups"), (dict(k=5, topk_groups=1), "fit"), (dict(group_topn=3), "group_topn"),
    (dict(bias=P + 2), "misaligned"), (dict(topk_idx=P + 1), "misaligned"), (dict(topk_prob=P + 2), "misaligned")])
def test_route_topk(kw, word):
    r, err = call("moe_route_topk", b.RouteTopkArgs, **{**TOPK, **kw})
    assert r == b.MGE_ERR_INVALID_ARG and word in err, err


@pytest.mark.parametrize("kw,word", [
    (dict(T=-1), "T"), (dict(E=300), "E"), (dict(k=9), "k"), (dict(score=-1), "score"), (dict(logits_dtype=7), "dtype"),
    (dict(logits_row_stride=1), "stride"), (dict(d_prob=None), "NULL"), (dict(d_logits=None), "NULL"),
    (dict(topk_idx=None), "NULL"), (dict(scale=float("nan")), "scale"), (dict(topk_idx=P + 2), "misaligned"),
    (dict(d_prob=P + 2), "misaligned"), (dict(d_logits=P + 1), "misaligned"), (dict(d_logits=P + 2, logits_dtype=1), "misaligned")])
def test_route_topk_bwd(kw, word):
    r, err = call("moe_route_topk_bwd", b.RouteTopkBwdArgs, **{**BWD, **kw})
    assert r == b.MGE_ERR_INVALID_ARG and word in err, err


def test_empty_calls_return_at_once():
    assert call("moe_route_topk", b.RouteTopkArgs, **{**TOPK, "T": 0, "logits": None, "topk_idx": None, "topk_prob": None})[0] == 0
    assert call("moe_route_topk_bwd", b.RouteTopkBwdArgs, **{**BWD, "T": 0, "logits": None, "topk_idx": None})[0] == 0
    assert call("mxfp4_quantize", b.Quant4Args, **{**QUANT, "R": 0, "in_": None})[0] == 0
    assert call("mxfp4_dequantize", b.Dequant4Args, rows=0, C=64)[0] == 0


QUANT = dict(batch=1, R=4, C=64, in_row_stride=64, in_=P, orient=3, row_codes=P, row_scales=P, col_codes=P, col_scales=P)


@pytest.mark.parametrize("kw,word", [
    (dict(C=48), "multiple of 32"), (dict(R=-1), "negative"), (dict(batch=-1), "negative"), (dict(batch=65536), "batch"),
    (dict(orient=0), "orient"), (dict(orient=4), "orient"), (dict(in_=None), "in must"), (dict(in_=P + 8), "aligned"),
    (dict(in_row_stride=63), "in_row_stride"), (dict(in_row_stride=68), "in_row_stride"),
    (dict(batch=2, in_batch_stride=64), "in_batch_stride"), (dict(R=65535 * 128 + 1, orient=1), "R must"),
    (dict(row_codes=None), "row"), (dict(row_scales=None), "row"), (dict(row_codes=P + 4), "row"),
    (dict(col_codes=None), "column"), (dict(col_scales=None), "column")])
def test_quantize4(kw, word):
    r, err = call("mxfp4_quantize", b.Quant4Args, **{**QUANT, **kw})
    assert r == b.MGE_ERR_INVALID_ARG and word in err, err


@pytest.mark.parametrize("kw", [dict(C=33), dict(rows=-1), dict(out_dtype=2), dict(codes=None), dict(codes=P + 1),
                                dict(scales=None), dict(out=None), dict(out=P + 2), dict(rows=1 << 40)])
def test_dequantize4(kw):
    base = dict(rows=4, C=64, out_dtype=0, codes=P, scales=P, out=P)
    assert call("mxfp4_dequantize", b.Dequant4Args, **{**base, **kw})[0] == b.MGE_ERR_INVALID_ARG


def gemm(**kw):
    w = (b.vp * 2)(P, P)
    bad = (b.vp * 2)(P, None)
    base = dict(a_format=0, E=2, N=64, K=64, rows=8, split_sizes=P, group_offsets=P, a=P, a_scale=P, out_dtype=0, out=P,
                w=C.cast(w, b.vp), w_scale=C.cast(w, b.vp), workspace=P, workspace_bytes=1 << 16)
    base.update({k: (C.cast(bad, b.vp) if v == "bad" else v) for k, v in kw.items()})
    return call("mxfp4_grouped_gemm", b.Gemm4Args, **base)


@pytest.mark.parametrize("kw,word", [
    (dict(a_format=2), "a_format"), (dict(E=0), "E"), (dict(E=257), "E"), (dict(N=48), "N and K"), (dict(K=0), "N and K"),
    (dict(K=80), "N and K"), (dict(rows=-1), "rows"), (dict(rows=1 << 26), "rows"), (dict(total_rows=-1), "total_rows"),
    (dict(N=1 << 22, K=1 << 10), "2^31"), (dict(split_sizes=None), "go together"), (dict(group_offsets=None), "go together"),
    (dict(split_sizes=None, group_offsets=None), "go together"), (dict(out_dtype=3), "out_dtype"), (dict(w=None), "NULL"),
    (dict(w="bad"), "expert 1"), (dict(w_scale="bad"), "expert 1"), (dict(a=None), "NULL"), (dict(a=P + 4), "misaligned"),
    (dict(a_scale=None), "NULL"), (dict(out=P + 8), "misaligned")])
def test_grouped_gemm4(kw, word):
    r, err = gemm(**kw)
    assert r == b.MGE_ERR_INVALID_ARG and word in err, err


def test_workspaces():
    assert gemm(workspace=None, rows=800)[0] == b.MGE_ERR_WORKSPACE
    assert gemm(workspace=None, rows=0)[0] == b.MGE_OK
    r, err = gemm(workspace_bytes=8, rows=800)
    assert r == b.MGE_ERR_WORKSPACE and "workspace needs" in err
    r, err = gemm(workspace=P + 8, workspace_bytes=1 << 24, rows=800)
    assert r == b.MGE_ERR_INVALID_ARG and "aligned" in err
    r, err = mlp(workspace=P + 8)
    assert r == b.MGE_ERR_INVALID_ARG and "aligned" in err
    assert b.lib().mge_gemm4_workspace_bytes(None) == 0
    assert b.lib().mge_fwd_mxfp4_workspace_bytes(None) == 0


def mlp(**kw):
    w = (b.vp * 2)(P, P)
    base = dict(prec=1, E=2, H=64, F=64, T=4, k=2, align=32, split_sizes=P, group_offsets=P, prob_perm=P, x_perm=P,
                x_perm_scale=P, y_perm=P, workspace=P, workspace_bytes=1 << 24)
    for n in ("w_gate_up", "w_gate_up_scale", "w_down", "w_down_scale"):
        base[n] = C.cast(w, b.vp)
    base.update(kw)
    return call("grouped_mlp_fwd_mxfp4", b.FwdArgs, **base)


def test_mlp4():
    assert mlp(prec=0)[0] == b.MGE_ERR_UNSUPPORTED
    for k in ("saved_gu", "h_col", "h_col_scale"):
        assert mlp(**{k: P})[0] == b.MGE_ERR_UNSUPPORTED
    for kw in (dict(x_perm_scale=None), dict(w_down_scale=None), dict(w_gate_up=None), dict(y_perm=P + 8), dict(h=P),
               dict(F=40), dict(H=0), dict(k=3), dict(align=3), dict(y_dtype=4), dict(prob_perm=None), dict(T=1 << 25)):
        assert mlp(**kw)[0] == b.MGE_ERR_INVALID_ARG, kw
    assert mlp(workspace_bytes=64)[0] == b.MGE_ERR_WORKSPACE
    assert mlp(T=0)[0] == b.MGE_OK


def test_python_checks():
    """Wrong dtypes, shapes and devices are refused before anything is allocated on a GPU."""
    import moe_grouped_expert_amd as m
    f = torch.zeros
    u8 = dict(dtype=torch.uint8)
    for fn in (lambda: m.moe_route_topk(f(4, 8), 2),                                    # not on a GPU
               lambda: m.moe_route_topk(f(4, 8, dtype=torch.float16), 2),
               lambda: m.moe_route_topk(f(4, 8), 2, score="relu"),
               lambda: m.moe_route_topk(f(8, 4).t(), 2),
               lambda: m.moe_route_topk_bwd(f(4, 8), f(4, 2, dtype=torch.int64), f(4, 2)),
               lambda: m.mxfp4_quantize(f(4, 64)),
               lambda: m.mxfp4_quantize(f(4, 64, dtype=torch.bfloat16), "rows"),
               lambda: m.mxfp4_quantize(f(64, 4, dtype=torch.bfloat16).t()),
               lambda: m.mxfp4_dequantize(f(4, 16, **u8), f(4, 2, **u8)),
               lambda: m.mxfp4_dequantize(f(4, 16, **u8), f(4, 1, **u8), "f16"),
               lambda: m.mxfp4_grouped_gemm(f(4, 48, **u8), f(4, 2, **u8), f(1, 32, 32, **u8), f(1, 32, 2, **u8)),
               lambda: m.mxfp4_grouped_gemm(f(4, 64, **u8), f(4, 2, **u8), f(1, 32, 16, **u8), f(1, 32, 2, **u8)),
               lambda: m.mxfp4_grouped_gemm(f(4, 64), f(4, 2, **u8), f(1, 32, 32, **u8), f(1, 32, 2, **u8))):
        with pytest.raises(ValueError):
            fn()


def test_python_route_without_activations():
    """An MXFP8 route made without x has nothing to multiply."""
    import moe_grouped_expert_amd as m
    z = torch.zeros(2, dtype=torch.int32)
    u8 = dict(dtype=torch.uint8)
    w, ws = torch.zeros(2, 64, 32, **u8), torch.zeros(2, 64, 2, **u8)
    for prec, x, xs in (("mxfp8", None, None), ("mxfp8", torch.zeros(32, 64, **u8), None), ("bf16", torch.zeros(32, 64), None)):
        rt = b.RouteOut(T=4, E=2, k=1, H=64, align=32, prec=prec, R=32, topk_idx=z, topk_prob=z, split_sizes=z, group_offsets=z,
                        perm_src=z, perm_pos=z, prob_perm=z, x_perm=x, x_perm_scale=xs)
        with pytest.raises(ValueError, match="route"):
            m.grouped_mlp_fwd_mxfp4(rt, w, w, ws, ws)
