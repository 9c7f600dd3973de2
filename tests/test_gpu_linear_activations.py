"""The projection's activations and their slopes on the GPU, value by value: one input of 1 and the
weights as arguments, so that z is exact."""
import numpy as np
import pytest
import torch

import gate_ref
import top_routing_expert_warp_b200 as moe

pytestmark = pytest.mark.gpu

TD = {"f32": torch.float32, "bf16": torch.bfloat16}
STEP = 2.0 ** -24          # half a step of fp32, relative
INF = float("inf")


def forward(act, z, dt, M):
    """act(z) in fp32 for every value of z, from M equal rows (which choose the kernel)."""
    N, K = len(z), 8
    cfg = moe.make_linear_config(M, K, N, act=act, dtype=dt, out_dtype="f32")
    ws = moe.linear_workspace(cfg)
    x, W = torch.zeros(M, K, dtype=TD[dt]), torch.zeros(N, K, dtype=TD[dt])
    x[:, 0], W[:, 0] = 1, z
    y = torch.empty(M, N, device="cuda")
    moe.moe_linear(cfg, x.cuda(), W.cuda(), None, None, y, None, ws)
    assert moe.moe_check_status(ws)[0] == moe.MOE_OK
    y = y.cpu()
    assert all(torch.equal(y[0], y[m]) for m in (M // 2, M - 1))
    return y[0].double().numpy()


def slope(act, z, dt):
    """act'(z) in fp32: the column sums of a single row."""
    N = len(z)
    cfg = moe.make_linear_config(1, 8, N, act=act, dtype=dt, out_dtype="f32")
    ws = moe.linear_workspace(cfg)
    db = torch.empty(N, device="cuda")
    moe.moe_linear_backward(cfg, torch.ones(1, N, device="cuda"), None, None, z.view(1, N).cuda(), None, None,
                            db, ws)
    return db.double().cpu().numpy()


def points(lo, hi, dt, n=4096):
    g = torch.Generator().manual_seed(1)
    z = torch.cat([torch.linspace(lo, hi, n - 64), torch.randn(64, generator=g) * 1e-3]).to(TD[dt])
    return z, z.double().numpy()


def normal_tail(z):
    """Phi(z) to 64 bits' relative precision on both sides."""
    from scipy.special import ndtr
    return ndtr(z)


KERNELS = [("f32", 1), ("f32", 8), ("bf16", 1), ("bf16", 16), ("bf16", 300)]


@pytest.mark.parametrize("dt,M", KERNELS)
def test_gelu_keeps_its_relative_precision(dt, M):
    """Phi(z) = e^{-z^2/2} r P(1 - 6 r), r = 1 / (|z| + 3): 9 steps of the polynomial, 3 for r, which
    enters twice, 6 for the exponential, 4 for products and the fit: below 32 half steps; and the
    exponent's own rounding, z^2 / 2 half steps."""
    z, zn = points(-12.5, 12.5, dt)
    want = zn * normal_tail(zn)
    assert np.all(np.abs(forward("gelu", z, dt, M) - want) <= (32 + zn * zn) * STEP * np.abs(want))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_gelu_slope_keeps_its_precision(dt):
    """The same of both terms, which cancel near -0.75."""
    z, zn = points(-12.5, 12.5, dt)
    phi, pdf = normal_tail(zn), np.exp(-zn * zn / 2) / np.sqrt(2 * np.pi)
    assert np.all(np.abs(slope("gelu", z, dt) - (phi + zn * pdf)) <=
                  (32 + zn * zn) * STEP * (phi + np.abs(zn) * pdf))


def test_gelu_near_zero():
    """Where most inputs lie: Phi off by less than 2e-7, so y by that times |z| and a rounding."""
    z, zn = points(-1.0, 1.0, "f32", 65536)
    want = zn * normal_tail(zn)
    assert np.all(np.abs(forward("gelu", z, "f32", 8) - want) <= np.abs(zn) * 2e-7 + STEP * np.abs(want))
