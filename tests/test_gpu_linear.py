"""The dense projection with its epilogue, and its gradients, on the GPU against 64-bit numpy."""
import numpy as np
import pytest
import torch

import gate_ref
import top_routing_expert_warp_b200 as moe

pytestmark = pytest.mark.gpu

TD = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}       # half a step, relative
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]
# rows, inputs, outputs, extra elements between rows
SHAPES = [(1, 8, 1, 0), (1, 1024, 264, 0), (2, 520, 130, 8), (7, 64, 33, 0), (16, 2048, 512, 0),
          (17, 72, 129, 16), (63, 136, 255, 0), (64, 4096, 64, 8), (100, 264, 96, 0),
          (129, 1032, 257, 8), (256, 256, 256, 0), (300, 520, 1000, 0), (513, 192, 520, 24),
          (1030, 328, 72, 0), (1000, 2056, 1500, 0), (2100, 520, 2561, 8), (40, 4096, 4096, 0), (640, 512, 384, 0),
          (384, 1024, 384, 0), (400, 648, 776, 8),
          (2100, 1400, 2561, 8), (9600, 1400, 72, 0)]


def strided(t, pad, fill=7.0):
    wide = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]], wide


def ints(g, *shape):
    return torch.randint(-3, 4, shape, generator=g)


def rounded(a, dtype):
    """64-bit values to the type, to nearest even."""
    t = torch.from_numpy(a)
    return t.float().to(TD[dtype]) if dtype == "bf16" else t.float()


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")], ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_linear_is_exact_on_whole_numbers(shape, types):
    """Products and sums of small whole numbers are exact in fp32, in every order: the outputs are
    the exact values, rounded once."""
    M, K, N, pad = shape
    dt, od = types
    g = torch.Generator().manual_seed(M + K)
    x, W, b, r = ints(g, M, K), ints(g, N, K), ints(g, N), ints(g, M, N)
    cfg = moe.make_linear_config(M, K, N, act="relu", dtype=dt, out_dtype=od, ldx=K + pad,
                                 ldy=N + pad + 1, ldr=N + 2 * pad)
    ws = moe.linear_workspace(cfg, backward=False)
    xd, _ = strided(x.to(TD[dt]).cuda(), pad)
    rd, _ = strided(r.to(TD[od]).cuda(), 2 * pad)
    y, wide = strided(torch.zeros(M, N, dtype=TD[od], device="cuda"), pad + 1, fill=5.0)
    z = torch.empty(M, N, dtype=TD[dt], device="cuda")
    moe.moe_linear(cfg, xd, W.to(TD[dt]).cuda(), b.float().cuda(), rd, y, z, ws)
    assert moe.moe_check_status(ws)[0] == moe.MOE_OK
    zz = x.double().numpy() @ W.double().numpy().T + b.double().numpy()
    assert torch.equal(z.cpu(), rounded(zz, dt))
    assert torch.equal(y.cpu(), rounded(np.maximum(zz, 0) + r.double().numpy(), od))
    assert torch.all(wide[:, N:] == 5.0)                     # between the rows nothing is written
    # without bias, residual and preact; and with the residual's place for y
    moe.moe_linear(cfg, xd, W.to(TD[dt]).cuda(), None, None, y, None, ws)
    assert torch.equal(y.cpu(), rounded(np.maximum(zz - b.double().numpy(), 0), od))
    same = moe.make_linear_config(M, K, N, act="relu", dtype=dt, out_dtype=od, ldx=K + pad,
                                  ldy=N + 2 * pad, ldr=N + 2 * pad)
    moe.moe_linear(same, xd, W.to(TD[dt]).cuda(), b.float().cuda(), rd, rd, None, ws)
    assert torch.equal(rd.cpu(), rounded(np.maximum(zz, 0) + r.double().numpy(), od))


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")], ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_linear_backward_is_exact_on_whole_numbers(shape, types):
    M, K, N, pad = shape
    dt, od = types
    g = torch.Generator().manual_seed(M + K + 1)
    x, W, dy, z = ints(g, M, K), ints(g, N, K), ints(g, M, N), ints(g, M, N)
    dz = (dy * (z > 0)).double().numpy()
    for act, grad in (("relu", dz), ("none", dy.double().numpy())):
        cfg = moe.make_linear_config(M, K, N, act=act, dtype=dt, out_dtype=od, ldx=K + pad, ldy=N + pad)
        ws = moe.linear_workspace(cfg)
        xd, _ = strided(x.to(TD[dt]).cuda(), pad)
        dyd, _ = strided(dy.to(TD[od]).cuda(), pad, fill=float("nan"))
        Wd = W.to(TD[dt]).cuda()
        zd = z.to(TD[dt]).cuda() if act == "relu" else None
        dx, wide = strided(torch.zeros(M, K, dtype=TD[dt], device="cuda"), pad, fill=5.0)
        dW = torch.empty(N, K, dtype=TD[dt], device="cuda")
        db = torch.empty(N, device="cuda")
        moe.moe_linear_backward(cfg, dyd, xd, Wd, zd, dx, dW, db, ws)
        assert moe.moe_check_status(ws)[0] == moe.MOE_OK
        wdx = rounded(grad @ W.double().numpy(), dt)
        wdW = rounded(grad.T @ x.double().numpy(), dt)
        wdb = rounded(grad.sum(0), "f32")
        assert torch.equal(dx.cpu(), wdx) and torch.equal(dW.cpu(), wdW) and torch.equal(db.cpu(), wdb)
        assert torch.all(wide[:, K:] == 5.0)
        # each output alone
        for i in range(3):
            out = [torch.empty_like(dW), torch.empty_like(db)]
            only, _ = strided(torch.zeros_like(dx), pad)
            moe.moe_linear_backward(cfg, dyd, xd if i == 1 else None, Wd if i == 0 else None, zd,
                                    only if i == 0 else None, out[0] if i == 1 else None,
                                    out[1] if i == 2 else None, ws)
            got, want = ((only, wdx), (out[0], wdW), (out[1], wdb))[i]
            assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")], ids=str)
@pytest.mark.parametrize("M", [1, 5, 40, 150])
@pytest.mark.parametrize("act", ACTS)
def test_linear_activations(act, M, types):
    K, N = 136, 200
    dt, od = types
    g = torch.Generator().manual_seed(M)
    x, W = torch.randn(M, K, generator=g).to(TD[dt]), (torch.randn(N, K, generator=g) * 0.3).to(TD[dt])
    b, r = torch.randn(N, generator=g), torch.randn(M, N, generator=g).to(TD[od])
    cfg = moe.make_linear_config(M, K, N, act=act, dtype=dt, out_dtype=od)
    ws = moe.linear_workspace(cfg)
    y, z = torch.empty(M, N, dtype=TD[od], device="cuda"), torch.empty(M, N, dtype=TD[dt], device="cuda")
    moe.moe_linear(cfg, x.cuda(), W.cuda(), b.cuda(), r.cuda(), y, z, ws)
    xn, Wn, bn = x.double().numpy(), W.double().numpy(), b.double().numpy()
    zz = xn @ Wn.T + bn
    # the sum: at most K + 1 steps, each off by a step (the tensor cores cut) of a partial sum
    ez = (K + 1) * 2.0 ** -23 * (np.abs(xn) @ np.abs(Wn).T + np.abs(bn))
    assert np.all(np.abs(z.double().cpu().numpy() - zz) <= ez + HALF[dt] * (np.abs(zz) + ez))
    want = gate_ref.act(act, zz)
    # the slope is at most 1.13, evaluating the function costs 16 half steps of |z| + 1
    ey = 1.13 * ez + 16 * 2.0 ** -24 * (np.abs(zz) + 1)
    want = want + r.double().numpy()
    ey = ey + 2.0 ** -24 * (np.abs(want) + np.abs(r.double().numpy()))
    assert np.all(np.abs(y.double().cpu().numpy() - want) <= ey + HALF[od] * (np.abs(want) + ey))


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")], ids=str)
@pytest.mark.parametrize("M", [1, 5, 40, 150])
@pytest.mark.parametrize("act", ACTS)
def test_linear_backward_activations(act, M, types):
    K, N = 136, 200
    dt, od = types
    g = torch.Generator().manual_seed(M + 1)
    x, W = torch.randn(M, K, generator=g).to(TD[dt]), torch.randn(N, K, generator=g).to(TD[dt])
    z, dy = (torch.randn(M, N, generator=g) * 3).to(TD[dt]), torch.randn(M, N, generator=g).to(TD[od])
    z[0, 0], z[0, 1], z[0, 2], z[0, 3] = 80.0, -80.0, 0.0, -12.0
    cfg = moe.make_linear_config(M, K, N, act=act, dtype=dt, out_dtype=od)
    ws = moe.linear_workspace(cfg)
    dx, dW = torch.empty(M, K, dtype=TD[dt], device="cuda"), torch.empty(N, K, dtype=TD[dt], device="cuda")
    db = torch.empty(N, device="cuda")
    moe.moe_linear_backward(cfg, dy.cuda(), x.cuda(), W.cuda(), None if act == "none" else z.cuda(),
                            dx, dW, db, ws)
    xn, Wn, zn, dyn = (t.double().numpy() for t in (x, W, z, dy))
    slope = gate_ref.act_grad(act, zn) if act != "none" else np.ones_like(zn)
    dz = dyn * slope
    # the slope in fp32: 32 half steps of |z| + 1 (its terms reach |z| / 4 and 1), at most 4 there
    # where |z| is not so large that they vanish; then dz's rounding to the operand type
    e32 = np.abs(dyn) * 32 * 2.0 ** -24 * (np.minimum(np.abs(zn), 20) + 1)
    ez = e32 + HALF[dt] * (np.abs(dz) + e32)
    for got, want, size, err, steps in (
            (dx, dz @ Wn, np.abs(dz) @ np.abs(Wn), ez @ np.abs(Wn), N),
            (dW, dz.T @ xn, np.abs(dz).T @ np.abs(xn), ez.T @ np.abs(xn), M)):
        tol = err + (steps + 1) * 2.0 ** -23 * size
        assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol + HALF[dt] * (np.abs(want) + tol))
    tol = e32.sum(0) + (M + 8) * 2.0 ** -24 * np.abs(dz).sum(0) + 1e-37
    assert np.all(np.abs(db.double().cpu().numpy() - dz.sum(0)) <= tol)


def test_linear_gradients_against_differences():
    """dx, dW and db against differences of the 64-bit projection."""
    M, K, N = 5, 16, 12
    g = torch.Generator().manual_seed(0)
    x, W, b = torch.randn(M, K, generator=g), torch.randn(N, K, generator=g) * 0.3, torch.randn(N, generator=g)
    dy = torch.randn(M, N, generator=g)
    cfg = moe.make_linear_config(M, K, N, act="gelu_tanh", dtype="f32")
    ws = moe.linear_workspace(cfg)
    y, z = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    dx, dW, db = torch.empty(M, K, device="cuda"), torch.empty(N, K, device="cuda"), torch.empty(N, device="cuda")
    moe.moe_linear(cfg, x.cuda(), W.cuda(), b.cuda(), None, y, z, ws)
    moe.moe_linear_backward(cfg, dy.cuda(), x.cuda(), W.cuda(), z, dx, dW, db, ws)
    xn, Wn, bn, dyn = (t.double().numpy() for t in (x, W, b, dy))
    rng, h = np.random.default_rng(1), 1e-6

    def loss(a, w, c):
        return (gate_ref.act("gelu_tanh", a @ w.T + c) * dyn).sum()
    for _ in range(5):
        ax, aw, ab = rng.normal(size=xn.shape), rng.normal(size=Wn.shape), rng.normal(size=bn.shape)
        num = (loss(xn + h * ax, Wn + h * aw, bn + h * ab) - loss(xn - h * ax, Wn - h * aw, bn - h * ab)) / (2 * h)
        parts = [(t.double().cpu().numpy() * a) for t, a in ((dx, ax), (dW, aw), (db, ab))]
        size = sum(np.abs(p).sum() for p in parts)
        # 64 half steps of each term; the difference itself is good to 1e-7 of the terms
        assert abs(num - sum(p.sum() for p in parts)) <= (64 * 2.0 ** -24 + 1e-7) * 4 * size


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_linear_empty_batch(dt):
    cfg = moe.make_linear_config(0, 16, 12, act="silu", dtype=dt)
    ws = moe.linear_workspace(cfg)
    e = lambda *s: torch.full(s, 3.0, dtype=TD[dt], device="cuda")  # noqa: E731
    moe.moe_linear(cfg, e(0, 16), e(12, 16), None, None, e(0, 12), None, ws)
    dW, db = e(12, 16), torch.full((12,), 3.0, device="cuda")
    moe.moe_linear_backward(cfg, e(0, 12), e(0, 16), e(12, 16), e(0, 12), e(0, 16), dW, db, ws)
    assert torch.all(dW == 0) and torch.all(db == 0)


@pytest.mark.parametrize("M", [1, 20, 300])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_linear_keeps_nan_and_inf_to_their_rows(dt, M):
    """A row with a NaN or an infinity spoils its own outputs only."""
    K, N = 264, 136
    g = torch.Generator().manual_seed(3)
    x, W = ints(g, M, K).to(TD[dt]), ints(g, N, K).to(TD[dt])
    x[M // 2, 5] = float("nan")
    cfg = moe.make_linear_config(M, K, N, act="none", dtype=dt, out_dtype="f32")
    ws = moe.linear_workspace(cfg)
    y = torch.empty(M, N, device="cuda")
    moe.moe_linear(cfg, x.cuda(), W.cuda(), None, None, y, None, ws)
    bad = torch.isnan(y).all(1).cpu()
    assert bad[M // 2] and bad.sum() == 1
    want = x.double() @ W.double().t()
    assert torch.equal(y.cpu()[~bad].double(), want[~bad])


@pytest.mark.parametrize("shape", [(1, 2048, 1000), (24, 4096, 300), (200, 4096, 129), (640, 512, 384),
                                   (384, 1024, 384), (512, 640, 640)], ids=str)
def test_linear_is_the_same_twice(shape):
    M, K, N = shape
    g = torch.Generator().manual_seed(1)
    x, W = torch.randn(M, K, generator=g).bfloat16().cuda(), torch.randn(N, K, generator=g).bfloat16().cuda()
    dy = torch.randn(M, N, generator=g).bfloat16().cuda()
    cfg = moe.make_linear_config(M, K, N)
    ws = moe.linear_workspace(cfg)
    seen = []
    for _ in range(2):
        y, dx, dW, db = (torch.empty_like(dy), torch.empty_like(x), torch.empty_like(W), torch.empty(N, device="cuda"))
        moe.moe_linear(cfg, x, W, None, None, y, None, ws)
        moe.moe_linear_backward(cfg, dy, x, W, None, dx, dW, db, ws)
        seen.append((y, dx, dW, db))
    assert all(torch.equal(a, b) for a, b in zip(*seen))


@pytest.mark.parametrize("shape", [(40, 4096, 1000), (600, 4096, 512), (4096, 4096, 2560), (9600, 4096, 72)],
                         ids=str)
def test_linear_fp32_results_are_summed_in_short_chains(shape):
    """fp32 results of bf16 operands: error of the norm at most 1.5e-6 (the tensor cores cut their
    sums at every step, 1e-9 of the norm per k of a chain; chains are at most 1280 long)."""
    M, K, N = shape
    g = torch.Generator().manual_seed(2)
    x, W = torch.randn(M, K, generator=g).bfloat16().cuda(), torch.randn(N, K, generator=g).bfloat16().cuda()
    cfg = moe.make_linear_config(M, K, N, out_dtype="f32")
    ws = moe.linear_workspace(cfg)
    y = torch.empty(M, N, device="cuda")
    moe.moe_linear(cfg, x, W, None, None, y, None, ws)
    want = x.double() @ W.double().t()
    assert ((y.double() - want).norm() / want.norm()).item() <= 1.5e-6


@pytest.mark.parametrize("M", [70001, 40])
def test_linear_rows_past_32_bit_offsets(M):
    """Rows 80 kB (or 132 MB) apart: element offsets past 2^31, on tiles of tokens and transposed."""
    K, N, ld = 64, 72, 40000 if M > 1000 else 66_000_000
    g = torch.Generator().manual_seed(5)
    x, W, r = ints(g, M, K).bfloat16(), ints(g, N, K).bfloat16(), ints(g, M, N).bfloat16()
    far = lambda t: torch.empty((M - 1) * ld + t.shape[1], dtype=t.dtype,  # noqa: E731
                                device="cuda").as_strided(t.shape, (ld, 1)).copy_(t)
    cfg = moe.make_linear_config(M, K, N, act="relu", ldx=ld, ldy=ld, ldr=ld)
    ws = moe.linear_workspace(cfg)
    xd, y = far(x), far(r)
    moe.moe_linear(cfg, xd, W.cuda(), None, y, y, None, ws)
    z = x.double().cuda() @ W.double().cuda().t()
    assert torch.equal(y, (z.clamp(min=0) + r.double().cuda()).bfloat16())
    dx, dW, db = far(x), torch.empty(N, K, dtype=torch.bfloat16, device="cuda"), torch.empty(N, device="cuda")
    flat = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    pre = z.bfloat16()
    moe.moe_linear_backward(cfg, y, xd, W.cuda(), pre, dx, dW, db, ws)
    assert moe.moe_check_status(ws)[0] == moe.MOE_OK
    dense = moe.make_linear_config(M, K, N, act="relu")
    dW2, db2 = torch.empty_like(dW), torch.empty_like(db)
    moe.moe_linear_backward(dense, y.contiguous(), x.cuda(), W.cuda(), pre, flat, dW2, db2, ws)
    assert torch.equal(dx, flat) and torch.equal(dW, dW2) and torch.equal(db, db2)
