"""GPU tests of the MXFP4 layer and products beside those of test_gpu_mxfp4.py: what a NaN does on its way through the
layer, more experts than a launch carries pointers for, h in the workspace, and the tail items of a product bit by bit."""
import dataclasses

import numpy as np
import pytest
import torch

from tests import test_gpu_mxfp4 as base
from tests.test_gpu_mxfp4 import layer, npy, operand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import moe_grouped_expert_amd as mge
    return mge


# tokens, experts, k, H, F: the streaming kernels, 64-row tiles, 256-row tiles of the gate-up product
PATHS = [(6, 4, 2, 128, 96), (40, 3, 2, 512, 160), (300, 4, 2, 384, 320), (2000, 3, 2, 256, 1056)]


@pytest.mark.parametrize("T,E,k,H,F", PATHS)
def test_nan_reaches_the_rows_it_belongs_to(m, T, E, k, H, F):
    """A NaN block of a weight (scale byte 255) makes every row of its expert NaN, one of a row of x that row, an E4M3
    NaN the same, and a row whose products overflow fp32 too; no other row changes a bit."""
    from tests.gpu_helpers import say
    say("[gpu] mlp4 nan", T, E, k, H, F)
    rt, (gc, gs, _, _), (dc, ds, _, _) = layer(m, T, E, k, H, F, T + E)
    valid = npy(rt.perm_src) >= 0
    ref = m.grouped_mlp_fwd_mxfp4(rt, gc, dc, gs, ds, y_dtype="f32")
    ref_y, ref_h, ref_s = ref.y_perm.clone(), ref.h.clone(), ref.h_scale.clone()
    sizes, off = npy(rt.split_sizes), npy(rt.group_offsets)
    e = int(sizes.argmax())
    o, n = int(off[e]), int(sizes[e])
    rows = np.arange(o, o + n)

    def run(hit, blocks):
        """hit: the rows that turn into NaN; blocks: whether only one block of 32 of their h does."""
        f = m.grouped_mlp_fwd_mxfp4(rt, gc, dc, gs, ds, y_dtype="f32")
        bad = np.zeros(rt.R, bool)
        bad[hit] = True
        keep = torch.from_numpy(valid & ~bad).cuda()
        assert np.isnan(npy(f.y_perm)[bad]).all()
        assert torch.equal(f.y_perm[keep], ref_y[keep]) and torch.equal(f.h[keep], ref_h[keep])
        assert torch.equal(f.h_scale[keep], ref_s[keep])
        s = npy(f.h_scale)[bad]
        if blocks is None:
            assert (s == 255).all()
        else:
            assert (s[:, blocks] == 255).all() and (np.delete(s, blocks, 1) != 255).all()

    for row, blk in ((F - 3, (F - 3) // 32), (F + 5, 0)):      # a gate row, an up row
        old = gs[e, row, 1].clone()
        gs[e, row, 1] = 255
        run(rows, blk)
        gs[e, row, 1] = old
    r = o + n // 2
    old = rt.x_perm_scale[r].clone()
    rt.x_perm_scale[r, H // 32 - 1] = 255
    run([r], None)
    rt.x_perm_scale[r] = 254                                   # |x| of 2^127 and more
    run([r], None)
    rt.x_perm_scale[r] = old
    old = rt.x_perm[r, 3].clone()
    rt.x_perm[r, 3] = 0x7F                                     # the E4M3 NaN
    run([r], None)
    rt.x_perm[r, 3] = old
    run([], None)


# streaming with the pointers in the arguments and in tables; 64-row tiles with both
MANY = [(9, 64, 2, 64, 32), (9, 65, 2, 64, 96), (30, 256, 8, 96, 64), (3300, 64, 2, 64, 64), (3300, 65, 2, 96, 64), (13000, 256, 2, 64, 32)]


@pytest.mark.parametrize("T,E,k,H,F", MANY)
def test_mlp_many_experts(m, T, E, k, H, F):
    """Against the 64-bit products, by the tolerances of test_mlp."""
    base.test_mlp(m, T, E, k, H, F, 8, None)


@pytest.mark.parametrize("T,E,k,H,F", [PATHS[0], PATHS[2], MANY[1], MANY[4]])
def test_mlp_with_h_in_the_workspace(m, T, E, k, H, F):
    """h = None: the same y, bit for bit, and a second call in the workspace of the first."""
    from tests.gpu_helpers import say
    say("[gpu] mlp4 without h", T, E, k, H, F)
    rt, (gc, gs, _, _), (dc, ds, _, _) = layer(m, T, E, k, H, F, T + 1)
    rows = torch.from_numpy(npy(rt.perm_src) >= 0).cuda()
    f = m.grouped_mlp_fwd_mxfp4(rt, gc, dc, gs, ds)
    g = dataclasses.replace(f, y_perm=torch.full_like(f.y_perm, 7.0), h=None, h_scale=None, workspace=None)
    assert m.grouped_mlp_fwd_mxfp4(rt, gc, dc, gs, ds, out=g) is g
    assert g.h is None and g.workspace.numel() >= rt.R * F
    assert torch.equal(g.y_perm[rows], f.y_perm[rows]) and bool((g.y_perm[~rows] == 7.0).all())
    ws = g.workspace
    g.y_perm.fill_(7.0)
    m.grouped_mlp_fwd_mxfp4(rt, gc, dc, gs, ds, out=g)
    assert g.workspace is ws and torch.equal(g.y_perm[rows], f.y_perm[rows])


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
def test_tail_items_equal_whole_tiles(m, fmt, out_dtype):
    """320 tiles of 256 x 256 are a whole round of 256 and 64 that run as quadrants; half of the columns are 160 tiles
    without a tail.  An element is summed in the same order in both: the same bits, of rounded data too."""
    from tests.gpu_helpers import say
    say("[gpu] gemm4 tail bits", fmt, out_dtype)
    rng = np.random.default_rng(31)
    sizes, N, K = [2100, 130], 8192, 288
    a, a_s, _ = operand(rng, sum(sizes), K, fmt, False)
    w, w_s, _ = operand(rng, 2 * N, K, "mxfp4", False)
    w, w_s = w.reshape(2, N, -1), w_s.reshape(2, N, -1)
    sz = torch.tensor(sizes, dtype=torch.int32, device="cuda")
    of = torch.tensor([0, sizes[0]], dtype=torch.int32, device="cuda")
    whole = m.mxfp4_grouped_gemm(a, a_s, w, w_s, sz, of, out_dtype)
    for lo in (0, N // 2):
        half = m.mxfp4_grouped_gemm(a, a_s, w[:, lo:lo + N // 2].contiguous(), w_s[:, lo:lo + N // 2].contiguous(), sz, of,
                                    out_dtype)
        assert torch.equal(whole[:, lo:lo + N // 2], half)
