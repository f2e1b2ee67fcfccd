"""GPU parity of rmsnorm_fwd and rmsnorm_bwd against the fp64 oracle.

Tolerances, with u = 2^-24 (fp32): a row's sum of squares is a sum of at most 64 terms a lane and 10 more joins, all
positive, so rstd is off by at most (74 / 2 + 6) u of itself and y by two roundings more; a result of n bits adds half a
step.  An 8-bit value is off by half a step, 2^-4 of itself or 2^-10 of its block's scale.  Of the backward's row mean
of g xhat the terms are rounded twice and the sum is off by at most 80 u of the sum of their magnitudes; a column of
dw adds at most ceil(T / 512) rows in a register, 3 waves, 32 parts and 16 slices."""
import numpy as np
import pytest
import torch

from oracle import fp8_block as fb

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": U}


@pytest.fixture(scope="module")
def m():
    import moe_grouped_expert_amd as mge
    return mge


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def rand(rng, shape, dt, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).cuda().to(DT[dt])


def check_fwd(m, T, H, xd="bf16", wd="bf16", res=True, form="fp8_block", yd="bf16", eps=1e-6, seed=0):
    from tests.gpu_helpers import say
    say("[gpu] rmsnorm", T, H, xd, wd, res, form, yd)
    rng = np.random.default_rng(seed + T + H)
    spread = np.exp(rng.standard_normal(H))
    x, r = rand(rng, (T, H), xd, spread), rand(rng, (T, H), xd, spread) if res else None
    w = rand(rng, H, wd)
    o = m.rmsnorm_fwd(x, w, eps, residual=r, form=form, y_dtype=yd)
    s = f64(x)
    if res:
        want = (x.float() + r.float()).to(DT[xd])
        assert torch.equal(o.residual, want)
        s = f64(want)
    else:
        assert o.residual is None
    y, rstd = fb.rmsnorm(s, f64(w), eps)
    assert np.all(np.abs(f64(o.rstd) - rstd) <= 44 * U * rstd)
    assert o.y.dtype == DT[yd]
    assert np.all(np.abs(f64(o.y) - y) <= (48 * U + HALF[yd]) * np.abs(y))
    if form is None:
        assert o.codes is None
        return
    amax = np.zeros((T, fb.blocks(H) * 128))
    amax[:, :H] = np.abs(y)
    amax = np.maximum(amax.reshape(T, -1, 128).max(2), 2.0 ** -100)
    sc = f64(o.scales)
    assert np.all(np.abs(sc * 448 - amax) <= 52 * U * amax)
    v = fb.decode(o.codes.cpu().numpy(), sc)
    step = np.maximum(np.abs(y) * 2.0 ** -4, fb.spread(sc, T, H, False) * 2.0 ** -10)
    assert np.all(np.abs(v - y) <= step * (1 + 2.0 ** -18) + 64 * U * np.abs(y))


@pytest.mark.parametrize("T,H", [(1, 32), (3, 96), (8, 4096), (33, 160), (2, 16384), (5, 8224), (257, 512), (2049, 544), (2100, 2080)])
@pytest.mark.parametrize("xd", ["bf16", "f32"])
def test_fwd(m, T, H, xd):
    check_fwd(m, T, H, xd, "bf16" if H % 64 else "f32")
    check_fwd(m, T, H, xd, "f32" if H % 64 else "bf16", res=False, yd="f32", seed=1)


def test_fwd_without_codes_or_y(m):
    check_fwd(m, 70, 1056, form=None)
    check_fwd(m, 70, 1056, "f32", "f32", form=None, yd="f32", res=False)
    rng = np.random.default_rng(4)
    x, w = rand(rng, (9, 192), "bf16"), rand(rng, 192, "bf16")
    o = m.rmsnorm_fwd(x, w, form="fp8_block", want_y=False)
    full = m.rmsnorm_fwd(x, w, form="fp8_block")
    assert o.y is None and torch.equal(o.codes, full.codes) and torch.equal(o.scales, full.scales)


def test_fwd_strides_shapes_and_in_place(m):
    rng = np.random.default_rng(5)
    wide, w = rand(rng, (40, 512), "bf16"), rand(rng, 256, "bf16")
    v = wide[:, 128:384]
    a, b = m.rmsnorm_fwd(v, w, form="fp8_block"), m.rmsnorm_fwd(v.contiguous(), w, form="fp8_block")
    for f in ("y", "codes", "scales", "rstd"):
        assert torch.equal(getattr(a, f), getattr(b, f))
    x, r = rand(rng, (2, 20, 256), "f32"), rand(rng, (2, 20, 256), "f32")
    a = m.rmsnorm_fwd(x, w, residual=r, form="fp8_block")
    assert a.y.shape == (2, 20, 256) and a.rstd.shape == (2, 20) and a.scales.shape == (2, 20, 2)
    keep = r.clone()
    out = m.RmsnormOut(y=torch.empty_like(a.y), residual=r)   # the stream is updated in place
    b = m.rmsnorm_fwd(x, w, residual=r, out=out)
    assert b is out and torch.equal(r, a.residual) and torch.equal(b.y, a.y) and not torch.equal(r, keep)
    e = m.rmsnorm_fwd(x[:, :0], w, form="fp8_block")
    assert e.y.shape == (2, 0, 256)


def test_fwd_bad_values_stay_in_their_row(m):
    rng = np.random.default_rng(6)
    x, w = rand(rng, (12, 288), "bf16"), rand(rng, 288, "bf16")
    ref = m.rmsnorm_fwd(x, w, form="fp8_block")
    y = x.clone()
    y[3, 7], y[5, 200], y[8] = float("nan"), float("inf"), 0
    got = m.rmsnorm_fwd(y, w, form="fp8_block")
    rows = [i for i in range(12) if i not in (3, 5, 8)]
    assert torch.equal(got.y[rows], ref.y[rows]) and torch.equal(got.codes[rows], ref.codes[rows]) and torch.equal(got.scales[rows], ref.scales[rows])
    assert torch.isnan(got.y[3]).all() and torch.isnan(got.scales[3]).all()
    assert torch.isnan(got.y[5, 200]) and not got.y[8].any() and not (got.codes[8] & 127).any()   # (signed zeros)
    assert torch.isfinite(got.scales[8]).all() and abs(got.rstd[8].item() - 1e3) < 1e-2
    # values far apart: the block scales differ by 2^60 and the small ones are kept
    z = torch.full((1, 256), 2.0 ** -30, device="cuda")
    z[0, :128] = 2.0 ** 30
    o = m.rmsnorm_fwd(z, torch.ones(256, device="cuda"), eps=0.0, form="fp8_block")
    v = fb.decode(o.codes.cpu().numpy(), o.scales.cpu().numpy())
    ref, _ = fb.rmsnorm(f64(z), np.ones(256), 0.0)
    assert np.all(np.abs(v - ref) <= ref * 64 * U)


def test_fwd_offsets_past_32_bits(m):
    T, H = 532480, 4096   # 2.2e9 values
    from tests.gpu_helpers import say
    say("[gpu] rmsnorm long", T, H)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(7)
    tail = rand(rng, (5, H), "bf16")
    x[-5:] = tail
    w = rand(rng, H, "bf16")
    o, ref = m.rmsnorm_fwd(x, w, form="fp8_block"), m.rmsnorm_fwd(tail, w, form="fp8_block")
    s = fb.rmsnorm(f64(tail), f64(w), 1e-6)[0]
    assert np.all(np.abs(f64(o.y[-5:]) - s) <= (48 * U + HALF["bf16"]) * np.abs(s))
    assert torch.equal(o.y[-5:], ref.y) or np.all(np.abs(f64(o.y[-5:]) - f64(ref.y)) <= 2.0 ** -7 * np.abs(s))
    assert not o.y[:-5].any()
    o.codes.bitwise_and_(127)   # (signed zeros)
    assert not o.codes[:-5].any()


def check_bwd(m, T, H, xd="bf16", wd="bf16", dyd="bf16", res=True, seed=0):
    from tests.gpu_helpers import say
    say("[gpu] rmsnorm_bwd", T, H, xd, wd, dyd, res)
    rng = np.random.default_rng(seed + T * 3 + H)
    x, w, dy = rand(rng, (T, H), xd, np.exp(rng.standard_normal(H))), rand(rng, H, wd), rand(rng, (T, H), dyd)
    dres = rand(rng, (T, H), xd) if res else None
    rstd = torch.from_numpy(fb.rmsnorm(f64(x), f64(w), 1e-6)[1].astype(np.float32)).cuda()
    dx, dw = m.rmsnorm_bwd(dy, x, w, rstd, d_residual=dres)
    rx, rw = fb.rmsnorm_bwd(f64(dy), f64(x), f64(w), f64(rstd))
    xhat = f64(x) * f64(rstd)[:, None]
    g = f64(dy) * f64(w)
    dot = np.abs((g * xhat).mean(-1, keepdims=True))
    near = f64(rstd)[:, None] * U * (8 * np.abs(g) + 8 * np.abs(xhat) * dot + 90 * np.abs(xhat) * np.abs(g * xhat).mean(-1, keepdims=True))
    d = f64(dres) if res else 0.0
    want = rx + d
    assert dx.dtype == DT[xd]
    assert np.all(np.abs(f64(dx) - want) <= (1 + HALF[xd]) * (near + 2 * U * (np.abs(rx) + np.abs(d))) + HALF[xd] * np.abs(want))
    mag = np.abs(f64(dy) * xhat).sum(0)
    assert np.all(np.abs(f64(dw) - rw) <= (-(-T // 512) + 56) * U * mag)


@pytest.mark.parametrize("T,H", [(1, 32), (3, 96), (8, 4096), (33, 160), (2, 16384), (5, 8224), (257, 512), (2049, 544), (2100, 2080), (1100, 1024)])
@pytest.mark.parametrize("xd", ["bf16", "f32"])
def test_bwd(m, T, H, xd):
    check_bwd(m, T, H, xd, "bf16" if H % 64 else "f32", "bf16")
    check_bwd(m, T, H, xd, "f32" if H % 64 else "bf16", "f32", res=False, seed=1)


def test_bwd_forms(m):
    rng = np.random.default_rng(8)
    wide = rand(rng, (300, 512), "bf16")
    x, dy, w = wide[:, :256], wide[:, 256:], rand(rng, 256, "bf16")
    rstd = m.rmsnorm_fwd(x, w).rstd
    a = m.rmsnorm_bwd(dy, x, w, rstd)
    b = m.rmsnorm_bwd(dy.contiguous(), x.contiguous(), w, rstd)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c = m.rmsnorm_bwd(dy, x, w, rstd, want_dw=False)
    assert c[1] is None and torch.equal(c[0], a[0])
    buf, dw = dy.contiguous(), torch.empty(256, device="cuda")
    d = m.rmsnorm_bwd(buf, x, w, rstd, out=(buf, dw))          # dx in dy's place
    assert d[0] is buf and torch.equal(buf, a[0]) and torch.equal(dw, a[1])
    e = m.rmsnorm_bwd(dy[:0], x[:0], w, rstd[:0], out=(x.new_empty(0, 256), dw.fill_(3.0)))
    assert not e[1].any()                                       # no rows: a zero gradient


def test_bwd_by_differences(m):
    """dx and dw against differences of the forward, in fp32: with a step h the forward's rounding is 64 u |y| / h."""
    rng = np.random.default_rng(9)
    T, H, h = 2, 64, 2.0 ** -6
    x, w, dy = rand(rng, (T, H), "f32"), rand(rng, H, "f32"), rand(rng, (T, H), "f32")
    o = m.rmsnorm_fwd(x, w, y_dtype="f32")
    dx, dw = m.rmsnorm_bwd(dy, x, w, o.rstd)
    loss = lambda a, b: (f64(m.rmsnorm_fwd(a, b, y_dtype="f32").y) * f64(dy)).sum()   # noqa: E731
    noise = 64 * U * np.abs(f64(o.y) * f64(dy)).sum() / h
    for i, j in [(0, 0), (0, 33), (1, 5), (1, 63)]:
        a, b = x.clone(), x.clone()
        a[i, j] += h
        b[i, j] -= h
        # (third derivative of a row's loss: below 32 |dy| |w| in units of the row's spread of one)
        assert abs((loss(a, w) - loss(b, w)) / (2 * h) - dx[i, j].item()) <= noise + 32 * h * h * float((dy[i] * w).abs().max())
    for j in (0, 17, 63):
        a, b = w.clone(), w.clone()
        a[j] += h
        b[j] -= h
        assert abs((loss(x, a) - loss(x, b)) / (2 * h) - dw[j].item()) <= noise   # linear in w


def test_captured_and_deterministic(m):
    rng = np.random.default_rng(10)
    x, r, w, dy = rand(rng, (3000, 1024), "bf16"), rand(rng, (3000, 1024), "bf16"), rand(rng, 1024, "bf16"), rand(rng, (3000, 1024), "bf16")

    def step():
        o = m.rmsnorm_fwd(x, w, residual=r, form="fp8_block")
        return [o.y, o.residual, o.codes, o.scales, o.rstd, *m.rmsnorm_bwd(dy, o.residual, w, o.rstd, d_residual=dy)]

    ref = [t.clone() for t in step()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for rep in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, out)), rep
        assert all(torch.equal(a, b) for a, b in zip(ref, step())), ("eager", rep)
    del graph


@pytest.mark.parametrize("T,H", [(700, 16384), (1500, 8192), (1700, 4096), (3000, 1056), (3001, 512), (3500, 1024)])
@pytest.mark.parametrize("xd", ["bf16", "f32"])
def test_bwd_several_rows_a_workgroup(m, T, H, xd):
    """More rows than workgroups: the next row on its way while one is reduced, and over a gradient in place."""
    check_bwd(m, T, H, xd, "bf16", "bf16")
    rng = np.random.default_rng(T)
    x, dy, dres, w = rand(rng, (T, H), xd), rand(rng, (T, H), xd), rand(rng, (T, H), xd), rand(rng, H, "f32")
    rstd = m.rmsnorm_fwd(x, w, y_dtype="f32").rstd
    dx, dw = m.rmsnorm_bwd(dy, x, w, rstd, dres)
    for i in range(3):
        args = [dy.clone(), x.clone(), w, rstd, dres.clone()]
        o = args[(0, 1, 4)[i]]
        got = m.rmsnorm_bwd(*args, out=(o, torch.empty_like(dw)))
        assert got[0] is o and torch.equal(o, dx) and torch.equal(got[1], dw), i
