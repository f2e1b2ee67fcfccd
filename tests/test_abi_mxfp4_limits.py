"""Limits of the MXFP4 calls (CPU): when a workspace is needed, and sizes past a launch."""
import ctypes as C
import os

import pytest

from moe_grouped_expert_amd import _binding as b
from tests import test_abi_topk_mxfp4 as base

pytestmark = pytest.mark.skipif(not os.path.exists(b.LIB_PATH), reason="libmge.so not built")


def many(fn, st, E, names, **kw):
    w = (b.vp * E)(*[base.P] * E)
    return base.call(fn, st, E=E, **{n: C.cast(w, b.vp) for n in names}, **kw)


@pytest.mark.parametrize("E,need", [(1, False), (64, False), (65, True), (256, True)])
@pytest.mark.parametrize("rows", [0, 1, 8])
def test_few_rows_need_a_workspace_past_64_experts(E, need, rows):
    """The weights' pointers travel with the launch for up to 64 experts, else in the workspace, empty calls included."""
    kw = dict(a_format=0, N=64, K=64, rows=rows, split_sizes=base.P, group_offsets=base.P, a=base.P, a_scale=base.P, out=base.P)
    g = b.Gemm4Args(struct_size=C.sizeof(b.Gemm4Args), E=E, **kw)
    assert (b.lib().mge_gemm4_workspace_bytes(C.byref(g)) > 0) == need
    if need:
        assert many("mxfp4_grouped_gemm", b.Gemm4Args, E, ("w", "w_scale"), **kw)[0] == b.MGE_ERR_WORKSPACE
    elif rows == 0:
        assert many("mxfp4_grouped_gemm", b.Gemm4Args, E, ("w", "w_scale"), **kw)[0] == b.MGE_OK
    kw = dict(prec=1, H=64, F=64, T=rows, k=1, align=32, split_sizes=base.P, group_offsets=base.P, prob_perm=base.P,
              x_perm=base.P, x_perm_scale=base.P, y_perm=base.P, h=base.P, h_scale=base.P)
    f = b.FwdArgs(struct_size=C.sizeof(b.FwdArgs), E=E, **kw)
    assert (b.lib().mge_fwd_mxfp4_workspace_bytes(C.byref(f)) > 0) == need
    names = ("w_gate_up", "w_gate_up_scale", "w_down", "w_down_scale")
    if need:
        assert many("grouped_mlp_fwd_mxfp4", b.FwdArgs, E, names, **kw)[0] == b.MGE_ERR_WORKSPACE
    elif rows == 0:
        assert many("grouped_mlp_fwd_mxfp4", b.FwdArgs, E, names, **kw)[0] == b.MGE_OK


@pytest.mark.parametrize("C_,ok", [(0x7fffff00, True), (0x7fffff20, False), (0x7fffffe0, False)])
def test_quantize_columns_past_a_launch(C_, ok):
    """A launch has 512 threads for 256 columns and fewer than 2^32 threads a row of workgroups; within the limit the
    call goes on to what its other arguments lack."""
    kw = {**base.QUANT, "R": 1, "C": C_, "in_row_stride": 1 << 31, "row_codes": None, "col_codes": None}
    r, err = base.call("mxfp4_quantize", b.Quant4Args, **kw)
    assert r == b.MGE_ERR_INVALID_ARG and ("row outputs missing" if ok else "C must be at most") in err, err


@pytest.mark.parametrize("rows,C_,ok", [((1 << 32) - 1024, 32, True), ((1 << 32) - 1023, 32, False), ((1 << 31) - 512, 64, True),
                                        ((1 << 31) - 511, 64, False)])
def test_dequantize_blocks_past_a_launch(rows, C_, ok):
    """A thread a block of 32 values; within the limit the call goes on to what its other arguments lack."""
    r, err = base.call("mxfp4_dequantize", b.Dequant4Args, rows=rows, C=C_, out_dtype=0, codes=base.P, scales=base.P, out=None)
    assert r == b.MGE_ERR_INVALID_ARG and ("NULL" if ok else "too many") in err, err


def test_python_workspaces_are_contiguous():
    """A strided workspace would be written between its elements too."""
    import torch

    import moe_grouped_expert_amd as m
    u8 = dict(dtype=torch.uint8)
    z, i = torch.zeros, torch.zeros(2, dtype=torch.int32)
    ws = z(1 << 16, 2, **u8)[:, 0]
    with pytest.raises(ValueError, match="workspace"):
        m.mxfp4_grouped_gemm(z(4, 64, **u8), z(4, 2, **u8), z(1, 32, 32, **u8), z(1, 32, 2, **u8), workspace=ws)
    rt = b.RouteOut(T=4, E=2, k=1, H=64, align=32, prec="mxfp8", R=66, topk_idx=i, topk_prob=i, split_sizes=i, group_offsets=i,
                    perm_src=i, perm_pos=i, prob_perm=i, x_perm=z(66, 64, **u8), x_perm_scale=z(66, 2, **u8))
    out = b.FwdOut(y_perm=z(66, 64, dtype=torch.bfloat16), h=None, workspace=ws)
    with pytest.raises(ValueError, match="workspace"):
        m.grouped_mlp_fwd_mxfp4(rt, z(2, 64, 32, **u8), z(2, 64, 16, **u8), z(2, 64, 2, **u8), z(2, 64, 1, **u8), out=out)
