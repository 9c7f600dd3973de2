"""The trainable gate on the GPU: routing of given logits, its gradient, the combine's gradient,
and a run of them together, against plain definitions in 64 bits (gate_ref)."""
import numpy as np
import pytest
import torch

import gate_ref
import oracle
import synth
import top_routing_expert_warp_b200 as moe

pytestmark = pytest.mark.gpu

TD = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}       # half a step, relative
INF = float("inf")


def strided(t, pad, fill=7.0):
    wide = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]], wide


def logits_of(T, N, seed, dtype, std=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, N, generator=g) * std).to(TD[dtype])


def run_route(l, bias, k, pad=0, score="softmax", p=True, **kw):
    T, N = l.shape
    dtype = "f32" if l.dtype is torch.float32 else "bf16"
    cfg = moe.make_route_config(T, N, k, score=score, dtype=dtype, ld=N + pad,
                                renormalize=kw.pop("renorm", False), **kw)
    ws = moe.route_workspace(cfg)
    x, _ = strided(l.cuda(), pad)
    idx = torch.full((T, k), -9, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -9.0, device="cuda")
    pm = torch.full((N,), -9.0, device="cuda") if p else None
    b = None if bias is None else bias.cuda()
    moe.moe_route(cfg, x, b, idx, w, pm, ws)
    status = moe.moe_check_status(ws)
    return idx.cpu().numpy(), w.cpu().numpy(), pm.cpu().numpy() if p else None, status


def check_route(l, bias, k, status=moe.MOE_OK, **kw):
    score = kw.get("score", "softmax")
    idx, w, p, st = run_route(l, bias, k, **kw)
    assert st[0] == status
    ref_kw = {n: v for n, v in kw.items() if n not in ("pad", "p")}
    b = None if bias is None else bias.numpy()
    ri, rw, rp = gate_ref.route(l.float().numpy(), b, k, **ref_kw)
    assert np.array_equal(idx, ri)
    # at most 16 fp32 operations of half a step each, on positive terms
    np.testing.assert_allclose(w, rw, rtol=2.0 ** -20, atol=1e-37)
    if p is not None:
        np.testing.assert_allclose(p, rp, rtol=2.0 ** -20, atol=1e-37)
    return score


GATES = {
    "sigmoid-nodes": dict(N=256, k=8, score="sigmoid", bias=0.05, renorm=True, scale=2.5,
                          n_groups=8, topk_groups=4, group_top=2),
    "softmax-nodes": dict(N=128, k=6, score="softmax", bias=None, renorm=True, scale=1.0,
                          n_groups=16, topk_groups=3, group_top=1),
    "softmax-nodes-bias": dict(N=96, k=4, score="softmax", bias=0.01, renorm=False, scale=16.0,
                               n_groups=4, topk_groups=2, group_top=3),
    "odd-nodes": dict(N=60, k=5, score="sigmoid", bias=0.2, renorm=False, scale=1.0,
                      n_groups=12, topk_groups=2, group_top=5),
    "deep-nodes": dict(N=240, k=8, score="softmax", bias=0.02, renorm=True, scale=1.0,
                       n_groups=3, topk_groups=1, group_top=60),
    "exact-fit": dict(N=64, k=8, score="sigmoid", bias=0.1, renorm=True, scale=1.0,
                      n_groups=16, topk_groups=2, group_top=4),      # as many experts as slots
    "top1": dict(N=128, k=1, score="softmax", bias=None, renorm=False, scale=1.0),
    "odd": dict(N=61, k=7, score="sigmoid", bias=0.1, renorm=True, scale=1.0),
    "few": dict(N=3, k=3, score="softmax", bias=1.0, renorm=True, scale=0.5),
    "one": dict(N=1, k=1, score="sigmoid", bias=None, renorm=False, scale=1.0),
    "wide-plain": dict(N=255, k=8, score="softmax", bias=None, renorm=False, scale=1.0),
}


@pytest.mark.parametrize("pad", [0, 3, 8])
@pytest.mark.parametrize("T", [1, 7, 333])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gate", list(GATES))
def test_route(gate, dtype, T, pad):
    kw = dict(GATES[gate])
    N, k, std = kw.pop("N"), kw.pop("k"), kw.pop("bias")
    l = logits_of(T, N, 11 * T + N, dtype)
    bias = None if std is None else torch.randn(N, generator=torch.Generator().manual_seed(5)) * std
    check_route(l, bias, k, pad=pad, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("nodes", [False, True])
def test_route_ties_and_near_ties(score, bias, nodes):
    """Equal values take the lowest index; values a 64-bit step or so apart in 32 bits are ordered
    as 64 bits order them."""
    T, N, k = 64, 64, 6
    g = torch.Generator().manual_seed(2)
    l = torch.randint(-2, 3, (T, N), generator=g).float()          # many exact ties
    l[16:32] = 0.0                                                  # a row of ties
    # neighbours one fp32 step apart, in shuffled places
    base = torch.full((32, N), 0.75)
    step = torch.stack([torch.randperm(N, generator=g) for _ in range(32)]).float()
    l[32:] = base + step * 2.0 ** -24
    # and a few of them near one another among others that are not
    l[48:, 5:] = torch.randn(16, N - 5, generator=g)
    b = None
    if bias:
        b = torch.zeros(N)
        b[N // 2:] = 2.0 ** -3
    kw = dict(n_groups=8, topk_groups=3, group_top=2) if nodes else {}
    check_route(l, b, k, score=score, renorm=True, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("nodes", [False, True])
@pytest.mark.parametrize("bias", [False, True])
def test_route_masked_and_extreme(score, nodes, bias):
    N, k = 64, 4
    l = logits_of(16, N, 9, "f32")
    l[0, :] = -INF                                   # nothing left
    l[1, :] = -INF
    l[1, 37] = 0.5                                   # one expert left
    l[2, 5:] = -INF                                  # five left, in the first node
    l[3, ::2] = -INF
    l[4, 10] = INF                                   # the largest finite value
    l[5, 10] = INF
    l[5, 50] = INF
    l[6, :] = torch.finfo(torch.float32).min         # the type's lowest value
    l[7, :] = torch.finfo(torch.float32).min
    l[7, 3] = 1.0
    l[8, :] = -90.0                                  # e^l is subnormal in fp32
    l[8, 20] = -89.0
    l[9, :] = 300.0
    l[10, :] = -0.0
    l[10, 1::2] = 0.0
    b = torch.randn(N, generator=torch.Generator().manual_seed(4)) * 0.1 if bias else None
    if bias:
        b[12] = -INF
        b[13] = INF
    kw = dict(n_groups=8, topk_groups=2, group_top=2) if nodes else {}
    if bias and score == "sigmoid":
        l = l[torch.arange(16) != 6]     # scores of exactly 0 with a bias: fine, but not equal logits
    for renorm in (False, True):
        check_route(l, b, k, score=score, renorm=renorm, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("nodes", [False, True])
@pytest.mark.parametrize("low", [-1e9, -3.0e38, -40.0])
def test_route_bias_that_masks_or_dwarfs_the_scores(low, nodes, score):
    """Experts held back by a large negative bias, and preferred by one far above the scores."""
    T, N, k = 400, 64, 6
    l = logits_of(T, N, 14, "f32")
    b = torch.randn(N, generator=torch.Generator().manual_seed(6)) * 0.05
    b[1::2] = low
    b[8] = 1000.0
    kw = dict(n_groups=8, topk_groups=3, group_top=2) if nodes else {}
    check_route(l, b, k, score=score, renorm=True, **kw)
    b[:] = low                                           # the scores are below the bias's last bit
    check_route(l, b, k, score=score, renorm=True, **kw)


def test_route_nan_counts_as_masked_and_is_reported():
    l = logits_of(9, 40, 1, "f32")
    l[3, 7] = float("nan")
    l[4, :] = float("nan")
    bias = torch.zeros(40)
    check_route(l, None, 3, status=moe.MOE_ERR_DEVICE_STATUS, score="sigmoid")
    bias[0] = float("nan")
    check_route(logits_of(9, 40, 1, "f32"), bias, 3, status=moe.MOE_ERR_DEVICE_STATUS)


def test_route_empty_batch_and_rows_behind():
    cfg = moe.make_route_config(0, 8, 2)
    ws = moe.route_workspace(cfg)
    e = lambda *s, **kw: torch.empty(*s, device="cuda", **kw)  # noqa: E731
    pm = torch.full((8,), 3.0, device="cuda")
    moe.moe_route(cfg, e(0, 8), None, e(0, 2, dtype=torch.int32), e(0, 2), pm, ws)
    assert torch.all(pm == 0)
    moe.moe_route_backward(cfg, e(0, 8), e(0, 2, dtype=torch.int32), e(0, 2), pm, e(0, 8), ws)
    # outputs longer than T rows: what lies behind stays
    T, N, k = 5, 40, 3
    cfg = moe.make_route_config(T, N, k, ld=N)
    ws = moe.route_workspace(cfg)
    l = logits_of(T, N, 3, "f32").cuda()
    idx = torch.full((T + 4, k), -3, dtype=torch.int32, device="cuda")
    w = torch.full((T + 4, k), -3.0, device="cuda")
    moe.moe_route(cfg, l, None, idx[:T], w[:T], None, ws)
    assert torch.all(idx[T:] == -3) and torch.all(w[T:] == -3) and torch.all(idx[:T] >= 0)
    dl = torch.full((T + 4, N), -3.0, device="cuda")
    moe.moe_route_backward(cfg, l, idx[:T], w[:T], None, dl[:T], ws)
    assert torch.all(dl[T:] == -3) and torch.all(torch.isfinite(dl[:T]))


def test_route_large_batch_is_the_same_twice():
    l = logits_of(20011, 256, 8, "f32")
    b = torch.randn(256, generator=torch.Generator().manual_seed(5)) * 0.05
    kw = dict(score="sigmoid", renorm=True, scale=2.5, n_groups=8, topk_groups=4, group_top=2)
    one, two = run_route(l, b, 8, **kw), run_route(l, b, 8, **kw)
    for a, c in zip(one[:3], two[:3]):
        assert np.array_equal(a, c)
    rows = slice(0, 20011, 97)
    ri, rw, _ = gate_ref.route(l.numpy()[rows], b.numpy(), 8, **kw)
    assert np.array_equal(one[0][rows], ri)
    np.testing.assert_allclose(one[1][rows], rw, rtol=2.0 ** -20)
    rp = gate_ref.shares(l.numpy(), "sigmoid").mean(0)
    np.testing.assert_allclose(one[2], rp, rtol=2.0 ** -20)


def grad_case(l, k, score, renorm, scale, seed, pad=0, dw=True, dp=True, idx=None):
    T, N = l.shape
    dtype = "f32" if l.dtype is torch.float32 else "bf16"
    g = torch.Generator().manual_seed(seed)
    dtw, dpm = torch.randn(T, k, generator=g), torch.randn(N, generator=g) * T
    if idx is None:
        idx = torch.stack([torch.randperm(N, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    cfg = moe.make_route_config(T, N, k, score=score, renormalize=renorm, scale=scale, dtype=dtype,
                                ld=N + pad)
    ws = moe.route_workspace(cfg)
    x, _ = strided(l.cuda(), pad)
    out, wide = strided(torch.zeros(T, N, dtype=l.dtype, device="cuda"), pad, fill=5.0)
    moe.moe_route_backward(cfg, x, idx.cuda() if dw else None, dtw.cuda() if dw else None,
                           dpm.cuda() if dp else None, out, ws)
    st = moe.moe_check_status(ws)
    if pad:
        assert torch.all(wide[:, N:] == 5.0)
    gg = dtw.double().numpy() if dw else np.zeros((T, k))
    cc = dpm.double().numpy() if dp else np.zeros(N)
    return out.double().cpu().numpy(), st, idx.long().numpy(), gg, cc


def close(got, want, tol):
    over = np.abs(got - want) - tol
    worst = np.unravel_index(np.argmax(over), over.shape)
    assert not over[worst] > 0, (worst, got[worst], want[worst], np.broadcast_to(tol, over.shape)[worst])
    assert not np.isnan(got).any()


def grad_tol(l, mag, dtype):
    """fp32: each term is a product of about 16 factors and sums of positive terms, each off by half
    a step, and of exponentials whose argument l - max is off by half a step of itself; then one
    rounding to the output type."""
    lc = np.where(np.isfinite(l), l, 0.0)
    arg = 2 * np.abs(lc).max()
    return (32 + 2 * arg) * 2.0 ** -24 * mag + (HALF[dtype] * mag if dtype == "bf16" else 0) + 1e-37


@pytest.mark.parametrize("parts", ["both", "dw", "dp"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("shape", [(1, 256, 8, 0), (333, 60, 4, 4), (50, 128, 1, 0), (33, 255, 8, 1),
                                   (9, 1, 1, 0), (200, 33, 5, 8)], ids=str)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_route_backward(dtype, shape, score, renorm, parts):
    T, N, k, pad = shape
    l = logits_of(T, N, T + N, dtype)
    got, st, idx, g, c = grad_case(l, k, score, renorm, 2.5, 3, pad, parts != "dp", parts != "dw")
    assert st[0] == moe.MOE_OK
    ln = l.double().numpy()
    want, mag = gate_ref.route_grad(ln, idx, g, c, score, renorm, 2.5)
    close(got, want, grad_tol(ln, mag, dtype))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_against_differences(score, renorm):
    T, N, k = 4, 12, 3
    l = logits_of(T, N, 21, "f32")
    got, _, idx, g, c = grad_case(l, k, score, renorm, 1.0, 4)
    ln, h = l.double().numpy(), 1e-6
    for t in range(T):
        for e in range(N):
            d = np.zeros_like(ln)
            d[t, e] = h
            num = (gate_ref.route_loss(ln + d, idx, g, c, score, renorm, 1.0) -
                   gate_ref.route_loss(ln - d, idx, g, c, score, renorm, 1.0)) / (2 * h)
            # sizes of order 1 here: the kernel within 64 half steps, the difference within 1e-7
            assert abs(num - got[t, e]) <= 64 * 2.0 ** -24 * max(1.0, np.abs(g).max() * 4) + 1e-7


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_masked_extreme_and_repeated(score, renorm):
    T, N, k = 8, 40, 3
    l = logits_of(T, N, 6, "f32")
    l[0, :] = -INF
    l[1, :] = -INF
    l[1, 4] = 0.25
    l[2, ::3] = -INF
    l[3, 5] = INF
    l[4, :] -= 95.0                     # scores are subnormal in fp32, their ratios are not
    g = torch.Generator().manual_seed(8)
    idx = torch.stack([torch.randperm(N, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    idx[1, 0] = 4
    idx[5] = torch.tensor([7, 7, 9])    # the same expert twice
    idx[6] = torch.tensor([8, 8, 8])
    got, st, _, gg, cc = grad_case(l, k, score, renorm, 1.0, 5, idx=idx)
    assert st[0] == moe.MOE_OK
    ln = l.double().numpy()
    want, mag = gate_ref.route_grad(ln, idx.long().numpy(), gg, cc, score, renorm, 1.0)
    off = np.isneginf(ln)
    assert np.all(got[off] == 0)
    assert np.all(np.isfinite(got))
    close(got, want, grad_tol(ln, mag, "f32"))


def test_route_backward_bad_index_and_nan_are_reported():
    l = logits_of(6, 20, 2, "f32")
    idx = torch.tensor([[0, 1], [-1, 2], [20, 3], [4, 5], [6, 7], [8, 9]], dtype=torch.int32)
    got, st, _, g, c = grad_case(l, 2, "sigmoid", False, 1.0, 7, idx=idx)
    assert st[0] == moe.MOE_ERR_DEVICE_STATUS
    ii = idx.long().numpy()
    g = np.where((ii < 0) | (ii >= 20), 0.0, g)          # left out
    want, mag = gate_ref.route_grad(l.double().numpy(), np.clip(ii, 0, 19), g, c, "sigmoid", False, 1.0)
    close(got, want, grad_tol(l.double().numpy(), mag, "f32"))
    l[2, 2] = float("nan")
    got, st, _, _, _ = grad_case(l, 2, "softmax", True, 1.0, 7)
    assert st[0] == moe.MOE_ERR_DEVICE_STATUS and np.all(np.isfinite(got)) and got[2, 2] == 0


# ------------------------------------------------------------------ the combine's gradient
SHAPES = [(1, 8, 8, 1), (5, 64, 8, 2), (40, 264, 16, 3), (33, 4104, 8, 2), (70, 2048, 16, 8),
          (300, 128, 16, 4), (17, 1032, 16, 5), (3, 12288, 16, 8)]


@pytest.mark.parametrize("cf", [0.0, 0.6])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_combine_backward(dtype, shape, cf):
    T, d, N, k = shape
    cfg = moe.make_config(T, d, N, k, 8, dtype=dtype, capacity_factor=cf)
    ws = moe.workspace(cfg)
    ref = oracle.dispatch(synth.synthetic_topk(3, T, N, k, skew=0.5), N, cf)
    g = torch.Generator().manual_seed(T + d)
    dy = torch.randn(T, d, generator=g).to(TD[dtype])
    yp = torch.randn(T * k, d, generator=g).to(TD[dtype])
    w = torch.rand(T, k, generator=g)
    inv = torch.from_numpy(ref["inv_row"])
    R = ref["R"]
    dyp = torch.full((T * k, d), 9.0, dtype=TD[dtype], device="cuda")
    dw = torch.full((T, k), 9.0, device="cuda")
    dev = [t.cuda() for t in (dy, yp, inv, w)]
    moe.moe_combine_backward(cfg, *dev, dyp, dw, ws)
    assert moe.moe_check_status(ws)[0] == moe.MOE_OK
    row = ref["inv_row"].reshape(T, k)
    dyn, ypn, wn = dy.double().numpy(), yp.double().numpy(), w.double().numpy()
    got, gotw = dyp.double().cpu().numpy(), dw.double().cpu().numpy()
    assert np.all(got[R:] == 9.0)                        # rows that no pair names
    for t in range(T):
        for j in range(k):
            r = row[t, j]
            if r < 0:
                assert gotw[t, j] == 0
                continue
            want = wn[t, j] * dyn[t]
            # one fp32 product, one rounding to the type
            assert np.all(np.abs(got[r] - want) <= (HALF[dtype] + 2.0 ** -23) * np.abs(want) + 1e-37)
            terms = dyn[t] * ypn[r]
            # a chain of at most d / 32 fused steps, then a tree over at most 1024 parts
            assert abs(gotw[t, j] - terms.sum()) <= (d / 32 + 16) * 2.0 ** -24 * np.abs(terms).sum()
    # one output alone, and in place
    only = torch.full((T, k), 9.0, device="cuda")
    moe.moe_combine_backward(cfg, dev[0], dev[1], dev[2], None, None, only, ws)
    assert torch.equal(only, dw)
    only = torch.full((T * k, d), 9.0, dtype=TD[dtype], device="cuda")
    moe.moe_combine_backward(cfg, dev[0], None, dev[2], dev[3], only, None, ws)
    assert torch.equal(only, dyp)
    place = dev[1].clone()
    dw2 = torch.empty_like(dw)
    moe.moe_combine_backward(cfg, dev[0], place, dev[2], dev[3], place, dw2, ws)
    assert torch.equal(dw2, dw) and torch.equal(place[:R], dyp[:R]) and torch.equal(place[R:], dev[1][R:])


def test_combine_backward_bad_rows_are_reported_and_left_out():
    T, d, k = 6, 64, 2
    cfg = moe.make_config(T, d, 8, k, 8, dtype="f32")
    ws = moe.workspace(cfg)
    inv = torch.arange(T * k, dtype=torch.int32)
    inv[3], inv[7] = T * k, -2
    yp = torch.ones(T * k, d, device="cuda")
    dyp, dw = torch.zeros(T * k, d, device="cuda"), torch.full((T, k), 9.0, device="cuda")
    moe.moe_combine_backward(cfg, torch.ones(T, d, device="cuda"), yp, inv.cuda(),
                             torch.ones(T, k, device="cuda"), dyp, dw, ws)
    assert moe.moe_check_status(ws)[0] == moe.MOE_ERR_DEVICE_STATUS
    bad = torch.zeros(T * k, dtype=torch.bool)
    bad[[3, 7]] = True
    assert torch.equal(dw.view(-1).cpu() == 0, bad) and torch.equal((dyp == 0).all(1).cpu(), bad)
    cfg = moe.make_config(0, d, 8, k, 8, dtype="f32")
    moe.moe_combine_backward(cfg, yp[:0], yp[:0], inv[:0].cuda(), dw[:0], dyp[:0], dw[:0],
                             moe.workspace(cfg))


def test_combine_backward_rows_past_32_bit_offsets():
    T, d, k = 70000, 8192, 4
    cfg = moe.make_config(T, d, 8, k, 8, dtype="bf16")
    ws = torch.zeros(moe.moe_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    dy = torch.full((T, d), 0.5, dtype=torch.bfloat16, device="cuda")
    yp = torch.full((T * k, d), 2.0, dtype=torch.bfloat16, device="cuda")        # 2.3e9 elements
    inv = torch.arange(T * k - 1, -1, -1, dtype=torch.int32, device="cuda")
    w = torch.arange(T * k, dtype=torch.float32, device="cuda").view(T, k) % 128
    dyp, dw = torch.zeros_like(yp), torch.empty(T, k, device="cuda")
    moe.moe_combine_backward(cfg, dy, yp, inv, w, dyp, dw, ws)
    assert moe.moe_check_status(ws)[0] == moe.MOE_OK
    assert torch.all(dw == d)                            # 8192 times 0.5 * 2
    want = (w.view(-1).flip(0) * 0.5).bfloat16()
    assert torch.equal(dyp[:, 0], want) and torch.equal(dyp[:, -1], want)


def test_route_rows_past_32_bit_offsets():
    T, N, k, ld = 70001, 64, 4, 20000                    # 5.6 GB from the first row to the last
    buf = torch.empty(T * ld, device="cuda").as_strided((T, N), (ld, 1))
    l = logits_of(T, N, 12, "f32")
    buf.copy_(l)
    cfg = moe.make_route_config(T, N, k, score="sigmoid", renormalize=True, ld=ld)
    ws = moe.route_workspace(cfg)
    idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    moe.moe_route(cfg, buf, None, idx, w, None, ws)
    dense = run_route(l, None, k, score="sigmoid", renorm=True, p=False)
    assert np.array_equal(idx.cpu().numpy(), dense[0]) and np.array_equal(w.cpu().numpy(), dense[1])
    dl = torch.empty(T * ld, device="cuda").as_strided((T, N), (ld, 1))
    moe.moe_route_backward(cfg, buf, idx, w, None, dl, ws)
    flat = torch.empty(T, N, device="cuda")
    moe.moe_route_backward(moe.make_route_config(T, N, k, score="sigmoid", renormalize=True), l.cuda(),
                           idx, w, None, flat, ws)
    assert torch.equal(dl, flat)


def test_route_on_a_given_stream():
    T, N, k = 300, 64, 4
    l = logits_of(T, N, 13, "f32")
    want = run_route(l, None, k)
    cfg = moe.make_route_config(T, N, k)
    x, ws = torch.zeros(T, N, device="cuda"), moe.route_workspace(cfg)
    idx, w = torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)                     # the copy ends long after the call returns
        x.copy_(l.cuda())
    moe.moe_route(cfg, x, None, idx, w, None, ws, stream=s)      # in order behind the copy
    s.synchronize()
    assert np.array_equal(idx.cpu().numpy(), want[0]) and np.array_equal(w.cpu().numpy(), want[1])


# ------------------------------------------------------------------ a run of them together
class GateStep:
    """One step of a layer with a trainable gate: projection to logits, routing, dispatch, experts,
    combine, and back to the gate's weights."""

    def __init__(self, T=200, d=256, N=32, k=4, H=128, seed=3):
        self.T, self.d, self.N, self.k = T, d, N, k
        g = torch.Generator().manual_seed(seed)
        bf = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).bfloat16().cuda()  # noqa: E731
        e = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
        i32, b16 = torch.int32, torch.bfloat16
        self.x, self.Wg = bf(T, d), bf(N, d, std=d ** -0.5)
        self.W1, self.W3, self.W2 = bf(N, H, d, std=d ** -0.5), bf(N, H, d, std=d ** -0.5), bf(N, d, H, std=H ** -0.5)
        self.dy = bf(T, d)
        self.bias = (torch.randn(N, generator=g) * 0.05).cuda()
        self.lc = moe.make_linear_config(T, d, N, dtype="bf16", out_dtype="f32")
        self.rc = moe.make_route_config(T, N, k, score="sigmoid", renormalize=True, scale=2.5,
                                        n_groups=4, topk_groups=2, group_top=2)
        self.cfg = moe.make_config(T, d, N, k, H, dtype="bf16", capacity_factor=4.0)
        self.lws, self.rws, self.ws = moe.linear_workspace(self.lc), moe.route_workspace(self.rc), moe.workspace(self.cfg)
        R = T * k
        self.logits, self.idx, self.w, self.p = e(T, N), e(T, k, dtype=i32), e(T, k), e(N)
        self.counts, self.offs, self.perm, self.inv = e(N, dtype=i32), e(N + 1, dtype=i32), e(R, dtype=i32), e(R, dtype=i32)
        self.drop, self.xp, self.yp = e(R, dtype=torch.uint8), e(R, d, dtype=b16), torch.zeros(R, d, dtype=b16, device="cuda")
        self.f, self.aux, self.y = e(N), e(1), e(T, d, dtype=b16)
        self.dw, self.dl, self.dyp = e(T, k), e(T, N), torch.zeros(R, d, dtype=b16, device="cuda")
        self.dx, self.dWg = e(T, d, dtype=b16), e(N, d, dtype=b16)

    def __call__(self):
        s = self
        moe.moe_linear(s.lc, s.x, s.Wg, None, None, s.logits, None, s.lws)
        moe.moe_route(s.rc, s.logits, s.bias, s.idx, s.w, s.p, s.rws)
        moe.moe_dispatch(s.cfg, s.x, s.idx, s.counts, s.offs, s.perm, s.inv, s.drop, s.xp, None, s.p,
                         s.f, s.aux, s.ws)
        moe.moe_expert_ffn(s.cfg, s.xp, None, s.offs, s.W1, s.W3, s.W2, s.yp, s.ws)
        moe.moe_combine(s.cfg, s.yp, s.inv, s.w, None, s.y, s.ws)
        moe.moe_combine_backward(s.cfg, s.dy, s.yp, s.inv, s.w, s.dyp, s.dw, s.ws)
        dp = s.f * (s.cfg.aux_alpha * s.N)
        moe.moe_route_backward(s.rc, s.logits, s.idx, s.dw, dp, s.dl, s.rws)
        moe.moe_linear_backward(s.lc, s.dl, s.x, s.Wg, None, s.dx, s.dWg, None, s.lws)

    def outputs(self):
        return [t.clone() for t in (self.y, self.idx, self.w, self.p, self.aux, self.dw, self.dl,
                                    self.dyp, self.dx, self.dWg)]

    def status(self):
        return [moe.moe_check_status(w)[0] for w in (self.lws, self.rws, self.ws)]


def test_gate_step_gradient_against_differences():
    s = GateStep()
    s()
    assert s.status() == [moe.MOE_OK] * 3
    x, Wg = s.x.double().cpu().numpy(), s.Wg.double().cpu().numpy()
    l = x @ Wg.T
    idx = s.idx.long().cpu().numpy()
    ri, _, _ = gate_ref.route(s.logits.cpu().numpy(), s.bias.cpu().numpy(), s.k, "sigmoid", True, 2.5, 4, 2, 2)
    assert np.array_equal(idx, ri)
    inv = s.inv.cpu().numpy().reshape(s.T, s.k)
    yp, dy = s.yp.double().cpu().numpy(), s.dy.double().cpu().numpy()
    dots = np.where(inv >= 0, (dy[:, None, :] * yp[np.maximum(inv, 0)]).sum(2), 0.0)
    assert np.any(inv < 0)                                  # some pairs over capacity
    c = s.cfg.aux_alpha * s.N * s.f.double().cpu().numpy()

    def loss(W):
        return gate_ref.route_loss(x @ W.T, idx, dots, c, "sigmoid", True, 2.5)
    dl, mag = gate_ref.route_grad(l, idx, dots, c, "sigmoid", True, 2.5)
    want, got = dl.T @ x, s.dWg.double().cpu().numpy()
    # logits' gradient rounded to bf16 (half a step of each), summed in fp32, rounded to bf16
    tol = 2.0 ** -8 * (mag.T @ np.abs(x)) + 2.0 ** -8 * np.abs(want)
    assert np.all(np.abs(got - want) <= tol)
    rng = np.random.default_rng(0)
    for _ in range(4):
        D = rng.normal(size=Wg.shape)
        h = 1e-5
        num = (loss(Wg + h * D) - loss(Wg - h * D)) / (2 * h)
        assert abs(num - (got * D).sum()) <= (tol * np.abs(D)).sum() + 1e-4 * abs(num)


def test_gate_step_captured_and_replayed():
    """The whole step captured into a graph, replayed on other inputs, equals the eager step; two
    graphs that share the workspaces replay in turn."""
    s = GateStep(seed=4)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        s()                                                  # first use outside the capture
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        s()
    with torch.cuda.graph(g2):
        s()
    other = GateStep(seed=5)
    for name in ("x", "Wg", "dy", "bias"):
        getattr(s, name).copy_(getattr(other, name))
    for name in ("W1", "W3", "W2"):
        getattr(s, name).copy_(getattr(other, name))
    other()
    want = other.outputs()
    R = int(other.offs[-1])
    for g in (g1, g2, g1):
        for t in (s.y, s.w, s.dl, s.dWg, s.dx):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = s.outputs()
        for i, (a, b) in enumerate(zip(got, want)):
            if i == 7:                                       # rows behind the kept ones are nobody's
                a, b = a[:R], b[:R]
            assert torch.equal(a, b), i
    assert s.status() == [moe.MOE_OK] * 3


def test_gate_steps_on_two_streams_at_once():
    a, b = GateStep(seed=6), GateStep(seed=7)
    a(), b()
    torch.cuda.synchronize()
    want = a.outputs(), b.outputs()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(sa):
            a()
        with torch.cuda.stream(sb):
            b()
    torch.cuda.synchronize()
    for s, w in ((a, want[0]), (b, want[1])):
        for x, y in zip(s.outputs(), w):
            assert torch.equal(x, y)
