"""Sizes at which byte offsets pass 2^31 or element counts 2^32: the norm, the quantizer, the products at their limits.  Most
of the data is zero and the rest small integers under powers of two, so that every sum is exact."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import moe_grouped_expert_amd as mge
    return mge


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    yield
    torch.cuda.empty_cache()


def say(*a):
    from tests.gpu_helpers import say as s
    s("[gpu] large", *a)


def codes_of(v):
    return v.to(torch.float8_e4m3fn).view(torch.uint8)


def sparse(rows, cols, seed, per_row=64):
    """Codes [rows, cols] with small integers at some places of every row, the first and the last column among them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.zeros(rows, cols, dtype=torch.uint8, device="cuda")
    at = torch.randint(0, cols, (rows, per_row), device="cuda", generator=g)
    at[:, 0], at[:, 1] = 0, cols - 1
    q.scatter_(1, at, codes_of(torch.randint(-3, 4, (rows, per_row), device="cuda", generator=g).float()))
    s = torch.exp2(torch.randint(-2, 3, (rows, (cols + 127) // 128), device="cuda", generator=g).float())
    return q, s


def value(q, s):
    return q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 1)[:, :q.shape[1]]


def tiles(N, K, seed):
    q, _ = sparse(N, K, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    return q, torch.exp2(torch.randint(-2, 3, ((N + 127) // 128, (K + 127) // 128), device="cuda", generator=g).float())


def tile_value(q, s, rows):
    """The values of some rows of a weight."""
    return q[rows].view(torch.float8_e4m3fn).double() * s[rows // 128].double().repeat_interleave(128, 1)[:, :q.shape[1]]


@pytest.mark.parametrize("rows", [40, 8191])
def test_long_rows_of_a(m, rows):
    """a of just under 2^31 bytes where there are many rows."""
    K, N = 1 << 18, 288
    say("gemm", rows, N, K)
    a, a_s = sparse(rows, K, 1)
    w, w_s = tiles(N, K, 2)
    out = m.fp8_block_grouped_gemm(a, a_s, w[None], w_s[None], out_dtype="f32")
    wv = tile_value(w, w_s, torch.arange(N, device="cuda"))
    for r in range(0, rows, 511):
        assert torch.equal(out[r].double(), wv @ value(a[r:r + 1], a_s[r:r + 1])[0]), r
    assert torch.equal(out[-1].double(), wv @ value(a[-1:], a_s[-1:])[0])


@pytest.mark.parametrize("rows", [3, 200])
def test_many_columns(m, rows):
    """2^22 columns: outputs of 2^31 bytes and more, a weight of 2^30."""
    K, N = 256, 1 << 22
    say("gemm", rows, N, K)
    a, a_s = sparse(rows, K, 3)
    w, w_s = tiles(N, K, 4)
    out = m.fp8_block_grouped_gemm(a, a_s, w[None], w_s[None], out_dtype="f32")
    av = value(a, a_s)
    for n0 in (0, 128 * 7 + 5, N // 2 - 100, N - 4096):
        n = torch.arange(n0, n0 + 4096 if n0 + 4096 <= N else N, device="cuda")
        assert torch.equal(out[:, n].double(), av @ tile_value(w, w_s, n).T.contiguous()), n0


def test_weight_gradient_of_many_tokens(m):
    """2^23 - 128 token columns, operands of just under 2^31 bytes."""
    R, N, K = (1 << 23) - 128, 256, 96
    say("wgrad", R, N, K)
    y, y_s = sparse(N, R, 5)
    x = torch.zeros(K, R, dtype=torch.uint8, device="cuda")
    x_s = torch.exp2(torch.randint(-2, 3, (K, R // 128), device="cuda").float())
    at = torch.cat([torch.arange(64, device="cuda"), torch.arange(R - 64, R, device="cuda"), torch.arange(64, device="cuda") * 131071])
    x[:, at] = codes_of(torch.randint(-3, 4, (K, len(at)), device="cuda").float())
    y[:, at] = codes_of(torch.randint(-3, 4, (N, len(at)), device="cuda").float())
    dw = m.fp8_block_grouped_wgrad(y, y_s, x, x_s)[0]
    at = at.unique()
    pick = lambda q, s: q[:, at].view(torch.float8_e4m3fn).double() * s[:, at // 128].double()   # noqa: E731
    assert torch.equal(dw.double(), pick(y, y_s) @ pick(x, x_s).T.contiguous())


def test_quantizer_past_32_bits(m):
    R, C = (1 << 17) + 160, 1 << 15
    say("quantize", R, C)
    x = torch.zeros(R, C, dtype=torch.bfloat16, device="cuda")
    for r in (0, R // 256 * 128, R - 160):
        x[r:r + 160].normal_()
    rc, rs, cc, cs = m.fp8_block_quantize(x, "both")
    for r in (0, R // 256 * 128, R - 160):
        n = min(160, R - r)
        a, b, c, d = m.fp8_block_quantize(x[r:r + n].contiguous(), "both")
        assert torch.equal(rc[r:r + n], a) and torch.equal(rs[r:r + n], b)
        if r % 128 == 0:      # (blocks of the transposed form begin at multiples of 128 rows)
            assert torch.equal(cc[:, r:r + 128], c[:, :128]) and torch.equal(cs[:, r // 128], d[:, 0])
    back = m.fp8_block_dequantize(rc, rs)
    assert torch.equal(back[-160:], m.fp8_block_dequantize(rc[-160:].contiguous(), rs[-160:].contiguous()))
    assert not back[1000:2000].any()


def test_norm_past_32_bits(m):
    T, H = (1 << 18) + 3, 16384
    say("norm", T, H)
    x = torch.full((T, H), 0.5, dtype=torch.bfloat16, device="cuda")
    x[-5:].normal_()
    w = torch.randn(H, device="cuda")
    o = m.rmsnorm_fwd(x, w, form="fp8_block")
    t = m.rmsnorm_fwd(x[-5:].contiguous(), w, form="fp8_block")
    assert torch.equal(o.y[-5:], t.y) and torch.equal(o.codes[-5:], t.codes) and torch.equal(o.scales[-5:], t.scales)
    assert torch.equal(o.y[1000], o.y[2000]) and torch.equal(o.y[T // 2], o.y[0])
    del o
    dx, dw = m.rmsnorm_bwd(x, x, w, torch.ones(T, device="cuda"), want_dw=False)
    u, _ = m.rmsnorm_bwd(x[-5:].contiguous(), x[-5:].contiguous(), w, torch.ones(5, device="cuda"), want_dw=False)
    assert dw is None and torch.equal(dx[-5:], u) and torch.equal(dx[T // 2], dx[0])
