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


def extremes(dt):
    z = torch.cat([torch.linspace(-100, -70, 500), torch.linspace(-30, -8, 500), torch.linspace(8, 100, 100),
                   torch.tensor([-1e4, -1e30, -3e38, 1e4, 1e18, 0.0])]).to(TD[dt])
    return z, z.double().numpy()


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("dt,M", KERNELS)
def test_activations_reach_their_limits(dt, M, act):
    """Far below 0 what is left is too small for fp32: the result is within 20 (100 for SiLU) of the
    smallest normal numbers of the value, and 0 at the end; far above it is the argument."""
    z, zn = extremes(dt)
    want = gate_ref.act(act, zn)
    if act == "gelu":
        want = zn * normal_tail(zn)                       # without the definition's cancellation
    if act == "gelu_tanh":
        from scipy.special import expit
        with np.errstate(over="ignore"):
            want = zn * expit(2 * np.sqrt(2 / np.pi) * (zn + 0.044715 * zn ** 3))
    y = forward(act, z, dt, M)
    # relative: 32 half steps, and the rounding of the exponents z, z^2 / 2 and 2 u (8 half steps of
    # the last's size, which has several operations)
    size = {"silu": 0 * zn, "relu": 0 * zn, "gelu": zn * zn / 2,
            "gelu_tanh": 8 * 1.6 * np.abs(zn + 0.044715 * zn ** 3)}[act]
    rel = (32 + np.minimum(size, 1000)) * STEP
    assert np.all(np.abs(y - want) <= rel * np.abs(want) + 100 * 2.0 ** -126)
    assert np.all(y[zn <= -1e4] == 0) and np.all(y[zn >= 1e4] == zn[zn >= 1e4])


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_slopes_reach_their_limits(dt, act):
    z, zn = extremes(dt)
    d = slope(act, z, dt)
    far = np.abs(zn) >= (90 if act == "silu" else 16)
    assert np.array_equal(d[far], (zn[far] > 0).astype(np.float64))
    assert np.all(np.isfinite(d))


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M", [1, 8])
def test_activations_of_infinities_and_nan(act, M):
    """Infinite and NaN sums, made by the bias: the functions' limits, and a NaN stays one."""
    cfg = moe.make_linear_config(M, 8, 3, act=act, dtype="f32")
    ws = moe.linear_workspace(cfg)
    y, z = torch.empty(M, 3, device="cuda"), torch.empty(M, 3, device="cuda")
    bias = torch.tensor([INF, -INF, float("nan")], device="cuda")
    moe.moe_linear(cfg, torch.ones(M, 8, device="cuda"), torch.ones(3, 8, device="cuda"), bias, None, y, z, ws)
    assert torch.all(y[:, 0] == INF) and torch.all(y[:, 1] == (-INF if act == "none" else 0))
    assert torch.all(torch.isnan(y[:, 2])) and torch.all(torch.isnan(z[:, 2]))
