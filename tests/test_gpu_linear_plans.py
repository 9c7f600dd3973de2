"""Products that the tensor-core planner cuts into three and four slices of k on CTA pairs (clusters
of six and eight), as the router's projection is: exact on whole numbers, in every direction."""
import numpy as np
import pytest
import torch

import top_routing_expert_warp_b200 as moe
from test_gpu_linear import TD, ints, rounded, strided

pytestmark = pytest.mark.gpu


def slices(rows, cols, k):
    """Slices on CTA pairs (0: not on pairs): tiles of 256 x 256, k in blocks of 64."""
    tiles, blocks = -(-rows // 256) * -(-cols // 256), -(-k // 64)
    if rows <= 128 or cols <= 128 or not (tiles >= 37 or tiles * blocks >= 592):
        return 0
    n = 1
    for m, held in ((2, 33), (3, 22), (4, 15)):
        n = m if tiles <= held and blocks >= 2 * m else n
    return n


# the product's rows, columns and k; 3 or 4 slices, the last columns and rows ragged
PRODUCTS = [(1201, 701, 2568, 4), (4097, 255, 2504, 3), (1537, 700, 1880, 3), (600, 1288, 2600, 3),
            (300, 200, 19008, 4), (129, 1537, 5440, 4)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("shape", PRODUCTS, ids=str)
def test_forward_in_slices_on_pairs(shape, out):
    M, N, K, n = shape
    assert slices(M, N, K) == n
    g = torch.Generator().manual_seed(M)
    x, W, b, r = ints(g, M, K), ints(g, N, K), ints(g, N), ints(g, M, N)
    for pad in (0, 8, 3):                                  # rows on 16-byte boundaries, and not
        cfg = moe.make_linear_config(M, K, N, act="relu", out_dtype=out, ldy=N + pad, ldr=N + pad)
        ws = moe.linear_workspace(cfg, backward=False)
        rd, _ = strided(r.to(TD[out]).cuda(), pad)
        y, wide = strided(torch.zeros(M, N, dtype=TD[out], device="cuda"), pad, fill=5.0)
        z = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        moe.moe_linear(cfg, x.bfloat16().cuda(), W.bfloat16().cuda(), b.float().cuda(), rd, y, z, ws)
        assert moe.moe_check_status(ws)[0] == moe.MOE_OK
        zz = (x.double().cuda() @ W.double().cuda().t()).cpu().numpy() + b.double().numpy()
        assert torch.equal(z.cpu(), rounded(zz, "bf16"))
        assert torch.equal(y.cpu(), rounded(np.maximum(zz, 0) + r.double().numpy(), out))
        assert torch.all(wide[:, N:] == 5.0)


@pytest.mark.parametrize("dy_type", ["bf16", "f32"])
@pytest.mark.parametrize("shape", PRODUCTS, ids=str)
@pytest.mark.parametrize("which", ["dx", "dW"])
def test_gradients_in_slices_on_pairs(which, shape, dy_type):
    I, J, L, n = shape
    J = -(-J // 8) * 8                                     # the inputs' width
    M, K, N = (I, J, L - 3) if which == "dx" else (L - 3, J, I)
    assert slices(I, J, L - 3) == n
    g = torch.Generator().manual_seed(M)
    x, W, dy = ints(g, M, K), ints(g, N, K), ints(g, M, N)
    pad = 0 if N % 2 else 5
    cfg = moe.make_linear_config(M, K, N, out_dtype=dy_type, ldy=N + pad, ldx=K + 8)
    ws = moe.linear_workspace(cfg)
    xd, _ = strided(x.bfloat16().cuda(), 8)
    dyd, _ = strided(dy.to(TD[dy_type]).cuda(), pad, fill=float("nan"))
    dx, wide = strided(torch.zeros(M, K, dtype=torch.bfloat16, device="cuda"), 8, fill=5.0)
    dW, db = torch.empty(N, K, dtype=torch.bfloat16, device="cuda"), torch.empty(N, device="cuda")
    moe.moe_linear_backward(cfg, dyd, xd, W.bfloat16().cuda(), None, dx, dW, db, ws)
    assert moe.moe_check_status(ws)[0] == moe.MOE_OK
    d = dy.double().cuda()
    assert torch.equal(dx, (d @ W.double().cuda()).float().bfloat16())
    assert torch.equal(dW, (d.t() @ x.double().cuda()).float().bfloat16())
    assert torch.equal(db, d.sum(0).float())
    assert torch.all(wide[:, K:] == 5.0)


@pytest.mark.parametrize("shape", [(1201, 701, 2568), (4097, 255, 2504)], ids=str)
def test_slices_on_pairs_are_the_same_twice(shape):
    M, N, K = shape
    g = torch.Generator().manual_seed(1)
    x, W = torch.randn(M, K, generator=g).bfloat16().cuda(), torch.randn(N, K, generator=g).bfloat16().cuda()
    cfg = moe.make_linear_config(M, K, N, act="gelu", out_dtype="f32")
    ws = moe.linear_workspace(cfg)
    one, two = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    moe.moe_linear(cfg, x, W, None, None, one, None, ws)
    moe.moe_linear(cfg, x, W, None, None, two, None, ws)
    assert torch.equal(one, two)
