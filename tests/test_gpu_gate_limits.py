"""Routing at the limits of its scores and masks, on the GPU against plain definitions in 64 bits
(gate_ref)."""
import numpy as np
import pytest
import torch

import gate_ref
import top_routing_expert_warp_b200 as moe

pytestmark = pytest.mark.gpu

INF = float("inf")


def run(l, bias, k, **kw):
    T, N = l.shape
    cfg = moe.make_route_config(T, N, k, dtype="f32" if l.dtype is torch.float32 else "bf16",
                                renormalize=kw.pop("renorm", False), **kw)
    ws = moe.route_workspace(cfg)
    idx = torch.full((T, k), -9, dtype=torch.int32, device="cuda")
    w, p = torch.full((T, k), -9.0, device="cuda"), torch.full((N,), -9.0, device="cuda")
    moe.moe_route(cfg, l.cuda(), None if bias is None else bias.cuda(), idx, w, p, ws)
    assert moe.moe_check_status(ws)[0] == moe.MOE_OK
    return idx.cpu().numpy(), w.cpu().numpy(), p.cpu().numpy()


def check(l, bias, k, **kw):
    idx, w, p = run(l, bias, k, **kw)
    ri, rw, rp = gate_ref.route(l.float().numpy(), None if bias is None else bias.numpy(), k, **kw)
    assert np.array_equal(idx, ri)
    # at most 16 fp32 operations of half a step each, on positive terms
    np.testing.assert_allclose(w, rw, rtol=2.0 ** -20, atol=1e-37)
    np.testing.assert_allclose(p, rp, rtol=2.0 ** -20, atol=1e-37)
    return p


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("N", [40, 128, 256])
@pytest.mark.parametrize("top", [2.0, -30.0, -59.0, -61.0])
def test_an_expert_off_in_every_row_has_no_share(top, N, score):
    g = torch.Generator().manual_seed(N)
    l = torch.rand(37, N, generator=g) * 4 + (top - 4)
    l[:, 7] = -INF
    l[:, N - 1] = -INF
    for bias in (None, torch.randn(N, generator=g) * 0.05):
        p = check(l, bias, 3, score=score)
        assert p[7] == 0 and p[N - 1] == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N", [40, 256])
def test_logistic_scores_far_below_the_rows_largest(N, dtype):
    """One row each, so that p is that row's shares: the largest logit is -59 and the others lie
    where e^l is near the smallest fp32 values, or are off."""
    g = torch.Generator().manual_seed(3)
    for low in (-70.0, -79.5, -81.0, -84.0, -86.0, -INF):
        l = torch.rand(1, N, generator=g) + low
        l[0, 9] = -59.0
        p = check(l.to(dtype), None, 3, score="sigmoid")
        if low == -INF:
            assert p[9] == 1.0 and np.count_nonzero(p) == 1


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("left", [0, 3, 7, 8, 9, 40])
@pytest.mark.parametrize("nodes", [False, True])
@pytest.mark.parametrize("by", ["bias", "logits"])
def test_few_experts_left_and_preferred_ones(by, nodes, left, score):
    """Fewer, just as many and a few more experts left than slots, some of them near ties, and
    biases of +inf: ranks, not the number of experts in sight, decide."""
    T, N, k = 65, 256, 8
    g = torch.Generator().manual_seed(left)
    l = torch.randn(T, N, generator=g)
    b = torch.randn(N, generator=g) * 0.05
    on = torch.randperm(N, generator=g)[:left]
    if left > 1:
        l[:, on[1]] = l[:, on[0]]                         # equal logits, biases one step apart
        b[on[1]] = torch.nextafter(b[on[0]], torch.tensor(1.0))
    off = torch.ones(N, dtype=torch.bool)
    off[on] = False
    if by == "bias":
        b[off] = -INF
    else:
        l[:, off] = -INF
    kw = dict(n_groups=8, topk_groups=4, group_top=2) if nodes else {}
    check(l, b, k, score=score, renorm=True, **kw)
    if left > 3:
        b[on[2:4]] = INF
        check(l, b, k, score=score, renorm=True, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_top", [1, 2, 4, 5])
@pytest.mark.parametrize("by", ["bias", "logits"])
def test_a_node_without_experts_scores_zero(by, group_top, score):
    """Its score is the sum of nothing: behind nodes with positive sums, ahead of negative ones."""
    T, N, G, k = 33, 64, 8, 6
    l = torch.randn(T, N, generator=torch.Generator().manual_seed(group_top))
    for shift in (0.5, -1.5):                             # all sums positive, all negative
        b = torch.full((N,), shift)
        b[40:48] += 0.25                                  # the fifth node ahead of the others
        x = l.clone()
        if by == "bias":
            b[16:24] = -INF
        else:
            x[:, 16:24] = -INF
        check(x, b, k, score=score, n_groups=G, topk_groups=1, group_top=group_top)
        idx, w, _ = run(x, b, k, score=score, n_groups=G, topk_groups=1, group_top=group_top)
        empty = (idx >= 16) & (idx < 24)
        assert empty.any() == (shift < 0)
        if by == "logits":
            assert np.all(w[empty] == 0)
        # a very low finite bias in place of -inf keeps the node behind all others
        b[16:24] = -1e30
        idx, _, _ = run(l, b, k, score=score, n_groups=G, topk_groups=1, group_top=group_top)
        assert not ((idx >= 16) & (idx < 24)).any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("nodes", [False, True])
@pytest.mark.parametrize("N", [64, 128, 256])
def test_many_equal_experts_before_a_slightly_better_one(N, nodes, score):
    """The first 40 experts are equal, and later ones better by less than 32 bits of the score show:
    the better ones are chosen, however many equal ones lie before them."""
    k = 4
    l = torch.full((24, N), 0.75)
    l[0, 50] += 2.0 ** -24                                # one fp32 step
    l[1, 41:] += 2.0 ** -24
    l[2] = 20.0                                           # logistic scores of 1 in 32 bits
    l[2, 45:52] = 22.0
    l[3, :] = 20.0
    l[3, 60] = INF
    l[4, :] = -30.0                                       # beside a bias that dwarfs them
    l[4, 55] = -29.0
    l[5, 40:] -= 2.0 ** -24                               # the first ones are the better ones
    l[7, ::3] = -INF                                      # equal, some off
    l[8, :] = -INF
    l[9, 3:40] = -INF
    l[9, 60] += 2.0 ** -24
    kw = dict(n_groups=4, topk_groups=3, group_top=2) if nodes else {}
    zero = torch.zeros(N)
    later = zero.clone()
    later[47] = 2.0 ** -30                                # the same by the bias
    for b in (zero, later, zero - 1.0, later - 1.0, zero + 1e6, torch.where(torch.arange(N) % 5 == 0, -INF, zero)):
        check(l, b, k, score=score, renorm=True, **kw)
