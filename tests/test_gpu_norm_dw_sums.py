"""The norm's weight gradient over many rows, against sums in 64 bits.

Tolerance, with u = 2^-24: x rstd is rounded once, and a product of dy and it joins its sum in one rounding.  A column's
sum adds the rows of a thread one after the other, ceil(T / n) of n workgroups or, where a wave has a row, ceil(T / 4n) and
then the other 3 waves; the n partial sums add up in 64 slices of ceil(n / 64), joined in 6 steps.  Every addition is off by
at most u of the sum of the magnitudes so far.  (n is what the workspace holds.)"""
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("T,H", [(40000, 8224), (24001, 16384), (30000, 8192), (40001, 2080), (60000, 1024), (60001, 512), (700, 1024)])
@pytest.mark.parametrize("xd", ["bf16", "f32"])
def test_dw_of_many_rows(T, H, xd):
    import moe_grouped_expert_amd as m
    from tests.gpu_helpers import say
    say("[gpu] rmsnorm_bwd dw", T, H, xd)
    g = torch.Generator(device="cuda")
    g.manual_seed(T + H)
    dt = torch.bfloat16 if xd == "bf16" else torch.float32
    # (a mean away from zero, so that sums grow with the rows)
    x = (torch.randn(T, H, generator=g, device="cuda") + 1).to(dt)
    dy = (torch.randn(T, H, generator=g, device="cuda") + 0.5).to(dt)
    w = torch.randn(H, generator=g, device="cuda")
    rstd = m.rmsnorm_fwd(x, w).rstd
    dw = m.rmsnorm_bwd(dy, x, w, rstd)[1].double()
    want, mag = torch.zeros(H, dtype=torch.float64, device="cuda"), torch.zeros(H, dtype=torch.float64, device="cuda")
    for i in range(0, T, 4096):
        p = dy[i:i + 4096].double() * (x[i:i + 4096].double() * rstd[i:i + 4096, None].double())
        want += p.sum(0)
        mag += p.abs().sum(0)
    n = m.lib().mge_rmsnorm_bwd_workspace_bytes(T, H) // (4 * H)
    wave = H <= 512 or (H <= 1024 and T >= 1024)
    adds = (-(-T // (4 * n)) + 3 if wave else -(-T // n)) + -(-n // 64) + 6
    assert torch.all((dw - want).abs() <= (adds + 1) * U * (1 + 2.0 ** -10) * mag)
