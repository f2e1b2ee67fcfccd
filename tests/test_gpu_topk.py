"""GPU parity of moe_route_topk and moe_route_topk_bwd against the fp64 oracle.

The choice is compared exactly.  Weights are fp32: with u = 2^-24, exp of an fp32 argument x
carries |x| u from the argument's own rounding and 2 u from the function, and a weight is one
exp, a sum of at most E of them (E/16 + 4 additions deep), a quotient and a product:
(E/16 + 16 + 2 max|l|) u relative bounds them all.  A gradient is a weight times
(d_i - sum_j w_j d_j) and for the sigmoid 1 - s_i: the same relative bound on
w_i (|d_i| + sum_j w_j |d_j|), and half a bf16 step where the gradient is bf16."""
import numpy as np
import pytest
import torch

from oracle import topk

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def m():
    import moe_grouped_expert_amd as mge
    return mge


def finite_max(l):
    f = np.abs(l[np.isfinite(l)])
    return float(f.max()) if f.size else 0.0


def check(m, l, k, score="softmax", bias=None, G=1, tg=1, topn=2, renorm=True, scale=1.0, bwd=True, seed=0):
    """l: a GPU tensor [T, E]."""
    from tests.gpu_helpers import npy, say
    T, E = l.shape
    say("[gpu] topk", T, E, k, score, "bias" if bias is not None else "", G, tg, topn, renorm, l.dtype)
    idx, prob = m.moe_route_topk(l, k, score=score, bias=bias, num_groups=G, topk_groups=tg, group_topn=topn,
                                 renormalize=renorm, scale=scale)
    ln = npy(l.float()).astype(np.float64)
    ref = topk.choose(ln, k, score, None if bias is None else npy(bias), G, tg, topn)
    np.testing.assert_array_equal(npy(idx), ref)
    w = topk.weights(ln, ref, score, renorm, scale)
    rel = (E / 16 + 16 + 2 * finite_max(ln)) * U
    assert np.all(np.abs(npy(prob) - w) <= rel * np.abs(w) + 1e-37)
    if not bwd:
        return
    rng = np.random.default_rng(seed + T)
    d = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    check_bwd(m, l, idx, d, score, renorm, scale)


def check_bwd(m, l, idx, d, score, renorm, scale):
    from tests.gpu_helpers import npy
    E = l.shape[1]
    got = m.moe_route_topk_bwd(l, idx, d, score=score, renormalize=renorm, scale=scale)
    assert got.dtype == l.dtype and got.shape == l.shape
    ln, ix, dn = npy(l.float()).astype(np.float64), npy(idx), npy(d).astype(np.float64)
    ref = topk.bwd(ln, ix, dn, score, renorm, scale)
    T, k = ix.shape
    mag = np.zeros_like(ref)
    for t in range(T):
        use = [i for i in range(k) if 0 <= ix[t, i] < E]
        if not use:
            continue
        w = topk.weights(ln[t:t + 1], ix[t:t + 1, use], score, renorm, 1.0)[0]
        tot = (w * np.abs(dn[t, use])).sum()
        for j, i in enumerate(use):
            mag[t, ix[t, i]] += abs(scale) * w[j] * (abs(dn[t, i]) + tot)
        if score == "softmax" and not renorm:
            mag[t] += abs(scale) * topk.scores(ln[t], score) * tot
    half = 0.0 if l.dtype == torch.float32 else 2.0 ** -8
    rel = (E / 16 + 24 + 2 * finite_max(ln)) * U
    g = npy(got.float()).astype(np.float64)
    assert np.all(np.abs(g - ref) <= half * np.abs(ref) + (1 + half) * rel * mag + 1e-37)


def logits(T, E, dtype, seed, masked=0.0, spread=1.5):
    rng = np.random.default_rng(seed)
    l = (spread * rng.standard_normal((T, E))).astype(np.float32)
    if masked:
        l[rng.random((T, E)) < masked] = -np.inf
        l[::7] = -np.inf                                   # nothing left
        l[3 % T] = -np.inf
        l[3 % T, E // 2] = 0.25                            # one expert left
    return torch.from_numpy(l).cuda().to(dtype)


def bias_of(E, seed):
    return torch.from_numpy((0.1 * np.random.default_rng(seed).standard_normal(E)).astype(np.float32)).cuda()


F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 2, 2), (3, 5, 5), (17, 16, 4), (33, 17, 8), (64, 60, 6), (130, 100, 8),
                                   (257, 129, 3), (300, 256, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_plain(m, T, E, k, score, dtype):
    check(m, logits(T, E, dtype, T + E), k, score, renorm=True, scale=2.5)
    check(m, logits(T, E, dtype, T + E + 1), k, score, bias=bias_of(E, E), renorm=False, scale=1.0)


@pytest.mark.parametrize("E,G,tg,k", [(256, 8, 4, 8), (256, 32, 3, 8), (60, 4, 2, 6), (30, 2, 1, 8), (12, 12, 5, 4), (8, 2, 1, 4),
                                      (255, 17, 4, 8), (200, 100, 7, 8)])
@pytest.mark.parametrize("topn", [1, 2])
@pytest.mark.parametrize("biased", [True, False])
def test_groups(m, E, G, tg, k, topn, biased):
    for i, (score, dtype, masked) in enumerate([("sigmoid", F32, 0.0), ("softmax", BF16, 0.2)]):
        check(m, logits(150, E, dtype, E + G + i, masked), k, score, bias_of(E, 9) if biased else None, G, tg, topn, True, 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("biased", [True, False])
def test_masks_and_ties(m, score, renorm, biased):
    b = bias_of(24, 1) if biased else None
    check(m, logits(80, 24, F32, 5, masked=0.5), 4, score, b, renorm=renorm)
    l = torch.round(logits(80, 24, F32, 6))                # many equal logits; -0 and +0
    l[::2] = l[::2] * 0.0
    check(m, l, 4, score, torch.zeros(24, device="cuda") if biased else None, 4, 2, 2, renorm)
    low = logits(40, 24, F32, 7)
    low[:, ::3] = torch.finfo(torch.float32).min           # a mask by the type's lowest value
    low[5] = torch.finfo(torch.float32).min
    check(m, low, 4, score, None, renorm=renorm, bwd=False) if score == "softmax" else None
    nan = logits(40, 24, F32, 8)
    nan[:, 3] = float("nan")
    check(m, nan, 4, score, b, renorm=renorm)


def test_extreme_sigmoids_keep_their_ratios(m):
    """All chosen scores underflow fp32: the renormalised weights are still those of the formula."""
    l = torch.tensor([[-200.0, -201.0, -203.0, -400.0], [-90.0, 5.0, -90.0, -91.0], [300.0, 299.0, -300.0, 1.0]], device="cuda")
    check(m, l, 3, "sigmoid", bwd=True)
    check(m, l, 2, "softmax", bwd=True)


def test_near_ties_rank_as_the_formula(m):
    """Keys 1e-9 apart, far below fp32 of the sums: the 64-bit choice."""
    rng = np.random.default_rng(12)
    T, E = 400, 32
    l = rng.standard_normal((T, E)).astype(np.float32)
    s = 1 / (1 + np.exp(-l.astype(np.float64)))
    bias = (1.0 - s[0]).astype(np.float32)                 # row 0: every key within fp32 rounding of 1
    l[1:200] = l[0] + (1e-6 * rng.standard_normal((199, E))).astype(np.float32)
    check(m, torch.from_numpy(l).cuda(), 8, "sigmoid", torch.from_numpy(bias).cuda(), 4, 2, 2, bwd=False)


@pytest.mark.parametrize("T,E,G,tg", [(300, 16, 4, 2), (300, 15, 3, 2), (3000, 64, 8, 3), (100, 64, 8, 3), (2500, 256, 8, 4), (100, 60, 4, 2)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_close_keys_everywhere(m, T, E, G, tg, score):
    """Rows of copies of few logits with biases a few fp32 steps apart: pairs, runs and whole groups of keys too close
    for fp32, in every token, at every width of the kernel."""
    rng = np.random.default_rng(T + E)
    l = rng.choice(rng.standard_normal(5).astype(np.float32), (T, E))
    l[: T // 3] = np.round(l[: T // 3])
    b = (0.25 + rng.integers(-3, 4, E) * 2.0 ** -24).astype(np.float32)
    for groups in ((1, 1), (G, tg)):
        check(m, torch.from_numpy(l).cuda(), 4, score, torch.from_numpy(b).cuda(), *groups, bwd=False)
        check(m, torch.from_numpy(l).cuda(), 4, score, None, *groups, bwd=False)


def test_bias_that_takes_experts_out(m):
    l = logits(50, 16, F32, 20)
    b = bias_of(16, 3)
    b[2], b[7], b[9] = -float("inf"), float("nan"), float("inf")
    from tests.gpu_helpers import npy
    idx, _ = m.moe_route_topk(l, 4, score="sigmoid", bias=b)
    ref = topk.choose(npy(l), 4, "sigmoid", npy(b))
    np.testing.assert_array_equal(npy(idx), ref)
    assert np.all(npy(idx)[:, 0] == 9) and not np.isin(npy(idx), [2, 7]).any()


def test_strided_rows_and_outputs(m):
    wide = logits(70, 300, F32, 30)
    for lo, E in ((0, 64), (3, 61), (8, 256)):             # aligned and not
        v = wide[:, lo:lo + E]
        check(m, v, 3, "sigmoid", bias_of(E, 4))
        out = (torch.empty(70, 3, dtype=torch.int32, device="cuda"), torch.empty(70, 3, device="cuda"))
        r = m.moe_route_topk(v, 3, out=out)
        assert r[0] is out[0] and torch.equal(r[0], m.moe_route_topk(v.contiguous(), 3)[0])
    wb = logits(70, 300, BF16, 31)
    check(m, wb[:, 1:130], 8, "softmax", None, 3, 2, 1)


def test_given_indices_backward(m):
    """A caller's own choice: repeated experts add up, indices outside [0, E) take no part."""
    l = logits(90, 20, F32, 40)
    rng = np.random.default_rng(41)
    idx = rng.integers(0, 20, (90, 5)).astype(np.int32)
    idx[::4, 1], idx[1::5, 2], idx[2::6, 0] = idx[::4, 0], 20, -1
    idx[10] = [-1, 20, 99, -5, 1 << 30]
    d = torch.from_numpy(rng.standard_normal((90, 5)).astype(np.float32)).cuda()
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            check_bwd(m, l, torch.from_numpy(idx).cuda(), d, score, renorm, 0.5)


def test_empty_and_one_long_call(m):
    z = torch.zeros(0, 8, device="cuda")
    idx, prob = m.moe_route_topk(z, 2)
    assert idx.shape == (0, 2) and m.moe_route_topk_bwd(z, idx, prob).shape == (0, 8)
    l = logits(20000, 64, F32, 50)
    a = m.moe_route_topk(l, 6, score="sigmoid", bias=bias_of(64, 5), num_groups=8, topk_groups=3)
    b = m.moe_route_topk(l[12345:12400], 6, score="sigmoid", bias=bias_of(64, 5), num_groups=8, topk_groups=3)
    assert torch.equal(a[0][12345:12400], b[0]) and torch.equal(a[1][12345:12400], b[1])


def test_same_as_the_router_of_the_permutation(m):
    """The softmax choice without bias or groups is moe_route_permute's own."""
    l = logits(500, 8, F32, 60)
    g = m.moe_route_permute(l, None, 2)
    idx, prob = m.moe_route_topk(l, 2)
    assert torch.equal(idx, g.topk_idx) and torch.allclose(prob, g.topk_prob, rtol=0, atol=2e-7)
    h = m.moe_route_permute(None, None, 2, E=8, topk_idx=idx, topk_prob=prob)
    assert torch.equal(h.perm_src, g.perm_src) and torch.equal(h.perm_pos, g.perm_pos)
