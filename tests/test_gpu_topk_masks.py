"""GPU parity of moe_route_topk and its backward where masks are the type's lowest value, choice, weights and gradients,
with the tolerances of test_gpu_topk.py over the logits that matter: such a logit is more than 1e30 below any other, its
score or ratio is exactly 0 in fp32 and in 64 bits, and between two of them the difference is exactly 0, so that none of
them adds to the argument's rounding."""
import numpy as np
import pytest
import torch

from tests import test_gpu_topk as base

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import moe_grouped_expert_amd as mge
    return mge


@pytest.mark.parametrize("T,E,k", [(40, 24, 4), (33, 60, 8), (2100, 256, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masks_of_the_lowest_value(m, monkeypatch, T, E, k, score, renorm, biased, dtype):
    monkeypatch.setattr(base, "finite_max", lambda l: float(np.abs(l[np.abs(l) < 1e30]).max()))
    l = base.logits(T, E, dtype, T + E)
    low = torch.finfo(dtype).min
    l[:, ::3] = low
    l[3, : E - 2] = low                                    # fewer left than are chosen
    l[5] = low                                             # none left
    l[7, 1::2] = -float("inf")                             # both kinds of masks
    b = base.bias_of(E, 2) if biased else None
    base.check(m, l, k, score, b, renorm=renorm)
    base.check(m, l, k, score, b, 4, 2, 2, renorm, 2.5)
