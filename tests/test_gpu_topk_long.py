"""moe_route_topk and its backward over more tokens than one launch takes: every token is reached, with the bits of a call
on its part alone."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,k", [((1 << 25) + 21, 8, 2), ((1 << 28) + 37, 2, 1)])
def test_more_tokens_than_a_launch(T, E, k):
    import moe_grouped_expert_amd as m
    from tests.gpu_helpers import say
    say("[gpu] topk long", T, E, k)
    g = torch.Generator(device="cuda").manual_seed(T % 1000)
    l = torch.empty(T, E, dtype=torch.bfloat16, device="cuda")
    d = torch.empty(T, k, device="cuda")
    step = 1 << 25
    for t in range(0, T, step):
        l[t:t + step].normal_(generator=g)
        d[t:t + step].normal_(generator=g)
    kw = dict(score="sigmoid", renormalize=False)
    idx = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    prob = torch.full((T, k), float("nan"), device="cuda")
    m.moe_route_topk(l, k, out=(idx, prob), **kw)
    dl = torch.full((T, E), float("nan"), dtype=torch.bfloat16, device="cuda")
    m.moe_route_topk_bwd(l, idx, d, out=dl, **kw)
    for t in range(0, T, step):
        s = slice(t, t + step)
        best = l[s].float().max(1).values
        assert torch.equal(l[s].float().gather(1, idx[s, :1].long())[:, 0], best), t
        if E == 2:
            assert torch.equal(idx[s, 0], (l[s, 1] > l[s, 0]).int()), t
        assert not bool(dl[s].isnan().any()) and not bool(prob[s].isnan().any()), t
        for a in (slice(max(t - 1500, 0), min(t + 1500, T)), slice(max(T - 3000, 0), T)):
            i, p = m.moe_route_topk(l[a], k, **kw)
            assert torch.equal(i, idx[a]) and torch.equal(p, prob[a]), (t, a)
            assert torch.equal(m.moe_route_topk_bwd(l[a], i, d[a], **kw), dl[a]), (t, a)
