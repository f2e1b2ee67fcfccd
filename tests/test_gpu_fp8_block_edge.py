"""Edges of the calls on FP8 with one fp32 scale per block of 128: rows of a group without a token, workspaces and outputs
of exactly their sizes, a bound of the rows that does not apply, the expert MLP's forms against each other."""
import numpy as np
import pytest
import torch

from oracle import fp8_block as fb
from tests.test_gpu_fp8_block import gpu, layer, npy, operand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import moe_grouped_expert_amd as mge
    return mge


# streamed, tiled with SwiGLU apart, tiled with SwiGLU in the product
@pytest.mark.parametrize("T,E,k,H,F", [(9, 4, 2, 160, 288), (300, 3, 2, 512, 768), (4100, 8, 2, 256, 1056)])
def test_mlp_rows_without_a_token(m, T, E, k, H, F):
    """perm_src outside x inside a group: rows of zeros; the other rows keep their bits."""
    from tests.gpu_helpers import say
    say("[gpu] mlp fb holes", T, E, k, H, F)
    rng = np.random.default_rng(T)
    x, x_s = (gpu(t) for t in fb.quantize(rng.standard_normal((T, H))))
    gu, gus, d, ds = layer(rng, E, H, F)
    w = [gpu(np.stack(t)) for t in (gu, d, [s[0] for s in gus], [s[0] for s in ds])]
    rt = m.moe_route_permute(gpu(rng.standard_normal((T, E)), np.float32), None, k, align=128)
    ref = m.grouped_mlp_fwd_fp8_block(rt, x, x_s, *w, y_dtype="f32")
    whole = npy(ref.y_perm).copy()
    off, sizes, src = npy(rt.group_offsets), npy(rt.split_sizes), npy(rt.perm_src).copy()
    inside = np.zeros(rt.R, bool)
    for o, n in zip(off, sizes):
        inside[o:o + n] = True
    rows = np.flatnonzero(inside)
    rows = rows[rng.random(len(rows)) < 0.3]
    src[rows] = rng.choice([-1, -7, T, T + 100, 2 ** 31 - 1], len(rows))
    rt.perm_src.copy_(gpu(src))
    got = npy(m.grouped_mlp_fwd_fp8_block(rt, x, x_s, *w, y_dtype="f32", out=ref).y_perm)   # over the first call's workspace
    hole = np.zeros(rt.R, bool)
    hole[rows] = True
    assert not got[hole].any()
    np.testing.assert_array_equal(got[inside & ~hole], whole[inside & ~hole])


@pytest.mark.parametrize("rows", [3, 40, 700])
def test_no_groups_take_every_row(m, rows):
    """Without groups all rows are one expert's, whatever total_rows says."""
    rng = np.random.default_rng(rows)
    a, a_s, av = operand(rng, rows, 160, True)
    w, w_s, wv = operand(rng, 288, 160, True, True)
    for total in (None, 1, rows):
        got = m.fp8_block_grouped_gemm(gpu(a), gpu(a_s), gpu(w)[None], gpu(w_s)[None], out_dtype="f32", total_rows=total)
        np.testing.assert_array_equal(npy(got), (av @ wv.T).astype(np.float32))


def guarded(n, dtype=torch.uint8):
    """A tensor of n elements inside a larger one of a known pattern, and a check of the pattern around it."""
    pad = 4096
    size = torch.empty(0, dtype=dtype).element_size()
    raw = torch.full((n * size + 2 * pad,), 0xA5, dtype=torch.uint8, device="cuda")
    view = raw[pad:pad + n * size].view(dtype)

    def check():
        assert bool((raw[:pad] == 0xA5).all()) and bool((raw[pad + n * size:] == 0xA5).all())
    return view, check


@pytest.mark.parametrize("sizes", [[3, 0, 1], [130, 7, 300]])
def test_products_stay_inside_their_buffers(m, sizes):
    from moe_grouped_expert_amd import _binding as b
    rng = np.random.default_rng(31)
    for E, N, K in ((3, 160, 288), (65, 32, 96)):
        sz = (sizes * E)[:E]
        off = np.cumsum([0] + [(n + 127) // 128 * 128 for n in sz])
        R = int(off[-1])
        a, a_s, _ = operand(rng, R, K, True)
        w, w_s, _ = zip(*(operand(rng, N, K, True, True) for _ in range(E)))
        want = m.fp8_block_grouped_gemm(gpu(a), gpu(a_s), gpu(np.stack(w)), gpu(np.stack(w_s)), gpu(sz, np.int32), gpu(off, np.int32))
        ga = b.GemmFbArgs(struct_size=b.C.sizeof(b.GemmFbArgs), E=E, N=N, K=K, rows=R, split_sizes=1, group_offsets=1)
        ws, ok_ws = guarded(b.lib().mge_gemm_fb_workspace_bytes(b.C.byref(ga)))
        out, ok_out = guarded(R * N, torch.bfloat16)
        m.fp8_block_grouped_gemm(gpu(a), gpu(a_s), gpu(np.stack(w)), gpu(np.stack(w_s)), gpu(sz, np.int32), gpu(off, np.int32),
                                 out=out.view(R, N), workspace=ws)
        ok_ws()
        ok_out()
        for n, o in zip(sz, off):
            assert torch.equal(out.view(R, N)[o:o + n], want[o:o + n])
        y, y_s, _ = operand(rng, N, R, True)
        x, x_s, _ = operand(rng, K, R, True)
        wa = b.WgradFbArgs(struct_size=b.C.sizeof(b.WgradFbArgs), E=E, N=N, K=K, rows=R)
        ws, ok_ws = guarded(b.lib().mge_wgrad_fb_workspace_bytes(b.C.byref(wa)))
        dw, ok_dw = guarded(E * N * K, torch.float32)
        m.fp8_block_grouped_wgrad(gpu(y), gpu(y_s), gpu(x), gpu(x_s), gpu(sz, np.int32), gpu(off, np.int32), out=dw.view(E, N, K), workspace=ws)
        ok_ws()
        ok_dw()


@pytest.mark.parametrize("R,C", [(1, 32), (33, 96), (129, 416)])
@pytest.mark.parametrize("block", ["1x128", "128x128"])
def test_quantizer_stays_inside_its_buffers(m, R, C, block):
    x = torch.randn(R, C, device="cuda").to(torch.bfloat16)
    want = m.fp8_block_quantize(x, "both", block)
    views, checks = zip(*(guarded(t.numel(), t.dtype) for t in want))
    got = m.fp8_block_quantize(x, "both", block, out=[v.view(t.shape) for v, t in zip(views, want)])
    for g, t, ok in zip(got, want, checks):
        ok()
        assert torch.equal(g, t)
    o, ok = guarded(R * C, torch.bfloat16)
    m.fp8_block_dequantize(want[0], want[1], out=o.view(R, C))
    ok()


def test_norm_stays_inside_its_buffers(m):
    for T, H in ((1, 32), (5, 160), (70, 4128), (3, 8224)):
        x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
        w = torch.randn(H, device="cuda")
        y, ok = guarded(T * H, torch.bfloat16)
        codes, ok_c = guarded(T * H)
        scales, ok_s = guarded(T * ((H + 127) // 128), torch.float32)
        rstd, ok_r = guarded(T, torch.float32)
        o = m.rmsnorm_fwd(x, w, form="fp8_block", out=m.RmsnormOut(y.view(T, H), codes.view(T, H), scales.view(T, -1), None, rstd))
        for c in (ok, ok_c, ok_s, ok_r):
            c()
        ref = m.rmsnorm_fwd(x, w, form="fp8_block")
        assert torch.equal(o.y, ref.y) and torch.equal(o.codes, ref.codes) and torch.equal(o.rstd, ref.rstd)


@pytest.mark.parametrize("T,H", [(0, 64), (1, 32), (3000, 64), (40, 16384)])
def test_extreme_sizes_of_the_norm(m, T, H):
    x = torch.randn(T, H, device="cuda")
    w = torch.randn(H, device="cuda")
    o = m.rmsnorm_fwd(x, w, y_dtype="f32")
    x64 = x.double()
    r = 1 / torch.sqrt((x64 ** 2).mean(1, keepdim=True) + 1e-6) if T else x64
    # the square's sum: H/256 additions in a thread and 12 across them; its root, quotient and two products 4 more
    tol = (H / 256 + 16) * 2.0 ** -24
    if T:
        assert bool(((o.y.double() - x64 * r * w.double()).abs() <= tol * (x64 * r * w.double()).abs() + 1e-30).all())
    dx, dw = m.rmsnorm_bwd(x, x, w, o.rstd if o.rstd is not None else torch.empty(T, device="cuda"))
    assert dx.shape == (T, H) and dw.shape == (H,)
    if T == 0:
        assert not dw.any()


def test_nothing_to_read(m):
    """Rows that a map sends to an operand without rows are zeros; a gated MLP of no tokens does nothing."""
    dev = "cuda"
    w, w_s = torch.full((2, 96, 160), 56, dtype=torch.uint8, device=dev), torch.ones(2, 1, 2, device=dev)
    none, none_s = torch.empty(0, 160, dtype=torch.uint8, device=dev), torch.empty(0, 2, device=dev)
    for sizes in ([3, 4], [300, 200]):
        n = sum(sizes)
        rows = gpu(np.arange(n), np.int32)
        got = m.fp8_block_grouped_gemm(none, none_s, w, w_s, gpu(sizes, np.int32), gpu([0, sizes[0]], np.int32), rows, out_dtype="f32")
        assert got.shape == (n, 96) and not got.any()
    wd, wd_s = torch.full((1, 160, 96), 56, dtype=torch.uint8, device=dev), torch.ones(1, 2, 1, device=dev)
    wg, wg_s = torch.full((1, 192, 160), 56, dtype=torch.uint8, device=dev), torch.ones(1, 2, 2, device=dev)
    assert m.grouped_mlp_fwd_fp8_block(None, none, none_s, wg, wd, wg_s, wd_s).y_perm.shape == (0, 160)


def test_two_graphs_and_eager_calls_between(m):
    """Two captured graphs and eager calls of other sizes share no workspace: every replay gives the eager bits."""
    rng = np.random.default_rng(41)
    w, w_s, _ = zip(*(operand(rng, 288, 416, False, True) for _ in range(3)))
    w, w_s = gpu(np.stack(w)), gpu(np.stack(w_s))
    calls = []
    for n in (9, 500):
        a, a_s, _ = operand(rng, n, 416, False)
        sizes = [n // 2, 0, n - n // 2]
        calls.append((gpu(a), gpu(a_s), w, w_s, gpu(sizes, np.int32), gpu(np.cumsum([0] + sizes[:2]), np.int32)))
    ref = [m.fp8_block_grouped_gemm(*c) for c in calls]
    x, nw = torch.randn(700, 416, device="cuda").to(torch.bfloat16), torch.randn(416, device="cuda")
    rs = m.rmsnorm_fwd(x, nw).rstd
    grad = m.rmsnorm_bwd(x, x, nw, rs, x)
    graphs, outs = [], []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append((m.fp8_block_grouped_gemm(*c), *m.rmsnorm_bwd(x, x, nw, rs, x)))
        graphs.append(g)
    for _ in range(3):
        for o in outs:
            for t in o:
                t.zero_()
        for g in graphs:
            g.replay()
        again = [m.fp8_block_grouped_gemm(*c) for c in calls]
        torch.cuda.synchronize()
        for o, r, e in zip(outs, ref, again):
            assert torch.equal(o[0], r) and torch.equal(e, r)
            assert torch.equal(o[1], grad[0]) and torch.equal(o[2], grad[1])
    graphs.clear()


def test_largest_value_of_a_block_is_the_largest_code(m):
    """Every mantissa of a block's largest value, at small, ordinary and the largest exponents: 448 / m rounded up or down,
    its code is E4M3's largest; in both orientations and in the norm, whose values are fp32."""
    bits = np.array([e * 128 + k for e in (0, 1, 20, 26, 27, 28, 64, 126, 127, 128, 200, 254) for k in range(128)], np.uint16)
    bits = bits[bits > 0]
    x = torch.from_numpy(bits.view(np.int16).copy()).cuda().view(torch.bfloat16)
    x = torch.stack([x, -x], 1).repeat_interleave(16, 1).contiguous()                # [n, 32]: m and -m
    for orient, t in (("row", x), ("col", x.t().contiguous())):
        t = t if orient == "row" else torch.nn.functional.pad(t, (0, -t.shape[1] % 32)).contiguous()
        got = m.fp8_block_quantize(t, orient)
        codes, scales = (got[0], got[1]) if orient == "row" else (got[2][:len(bits)], got[3][:len(bits)])
        q, s = fb.quantize(x.float().cpu().numpy())
        np.testing.assert_array_equal(npy(codes)[:, :32], q)
        np.testing.assert_array_equal(npy(scales), s)
    big = bits >= 28 * 128
    assert (q[big] & 127 == 126).all()
    g = torch.Generator(device="cuda").manual_seed(5)
    v = torch.rand(4096, 128, device="cuda", generator=g) + 0.5
    o = m.rmsnorm_fwd(v, torch.ones(128, device="cuda"), form="fp8_block", y_dtype="f32")
    q, s = fb.quantize(npy(o.y))
    np.testing.assert_array_equal(npy(o.codes), q)
    np.testing.assert_array_equal(npy(o.scales), s)
