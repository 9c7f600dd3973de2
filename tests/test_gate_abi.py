"""The gate's and the projection's entry points refuse bad arguments on the host, before any
launch, and the plain definitions the GPU tests compare with agree with differences (no GPU)."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import gate_ref
import top_routing_expert_warp_b200 as moe
from top_routing_expert_warp_b200 import build as moe_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 40          # never dereferenced: validation fails first
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.lib()


@pytest.mark.parametrize("struct", ["moe_route_config", "moe_linear_config"])
def test_structs_match_their_ctypes_mirrors(struct):
    txt = open(os.path.join(ROOT, "include", "moe.h")).read()
    body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (struct, struct), txt, flags=re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    ct = {"int64_t": ctypes.c_int64, "int32_t": ctypes.c_int32, "float": ctypes.c_float}
    fields = [(n, ct[t]) for t, n in re.findall(r"\b(int64_t|int32_t|float)\s+(\w+);", body)]
    assert fields == list(getattr(moe, struct)._fields_)


ROUTE = dict(T=16, N=64, k=4, score="sigmoid")
BAD_ROUTE = [dict(N=0), dict(N=257), dict(k=0), dict(k=9), dict(N=3), dict(T=-1), dict(T=1 << 30),
             dict(ld=63), dict(n_groups=7, topk_groups=2, group_top=1),      # 64 % 7
             dict(n_groups=64, topk_groups=8, group_top=1),                  # over 32 nodes
             dict(n_groups=32, topk_groups=1, group_top=1),                  # 2 experts for k = 4
             dict(n_groups=8, topk_groups=0, group_top=1), dict(n_groups=8, topk_groups=2),
             dict(n_groups=8, topk_groups=2, group_top=9), dict(n_groups=-1), dict(topk_groups=-1),
             dict(group_top=-1), dict(scale=float("inf")), dict(scale=float("nan"))]


@pytest.mark.parametrize("bad", BAD_ROUTE, ids=str)
def test_route_config_refusals(lib, bad):
    good = moe.make_route_config(**ROUTE)
    assert moe.moe_route_workspace_bytes(good) > 0
    cfg = moe.make_route_config(**{**ROUTE, **bad})
    assert moe.moe_route_workspace_bytes(cfg) == 0
    a = [P(FAKE)] * 6
    assert lib.moe_route(ctypes.byref(cfg), *a, 1 << 40, None) == moe.MOE_ERR_INVALID_ARG
    assert lib.moe_route_backward(ctypes.byref(cfg), *a, 1 << 40, None) == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("field,value", [("score", 2), ("renormalize", 2), ("dtype", 2),
                                         ("dtype", -1)])
def test_route_enum_refusals(lib, field, value):
    cfg = moe.make_route_config(**ROUTE)
    setattr(cfg, field, value)
    assert moe.moe_route_workspace_bytes(cfg) == 0


def test_route_argument_refusals(lib):
    cfg = moe.make_route_config(**ROUTE)
    n = moe.moe_route_workspace_bytes(cfg)
    c = ctypes.byref(cfg)
    inv, wsp = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_WORKSPACE
    ok = [P(FAKE), None, P(FAKE), P(FAKE), None]

    def route(args=ok, ws=P(FAKE), nb=n):
        return lib.moe_route(c, *args, ws, nb, None)
    for i in (0, 2, 3):                                       # required
        assert route([None if j == i else a for j, a in enumerate(ok)]) == inv
    for i in range(5):                                        # misaligned
        assert route([P(FAKE + 2) if j == i else a for j, a in enumerate(ok)]) == inv
    assert route(ws=None) == wsp and route(ws=P(FAKE + 8)) == wsp and route(nb=n - 1) == wsp

    ok2 = [P(FAKE), P(FAKE), P(FAKE), None, P(FAKE + 4096)]

    def back(args=ok2, ws=P(FAKE), nb=n):
        return lib.moe_route_backward(c, *args, ws, nb, None)
    for i in (0, 1, 4):                                       # topk_idx goes with dtopk_w
        assert back([None if j == i else a for j, a in enumerate(ok2)]) == inv
    for i in range(5):
        assert back([P(FAKE + 2) if j == i else a for j, a in enumerate(ok2)]) == inv
    assert back(ok2[:4] + [P(FAKE)]) == inv                   # in place
    assert back(ws=None) == wsp and back(ws=P(FAKE + 8)) == wsp and back(nb=n - 1) == wsp


def test_combine_backward_argument_refusals(lib):
    cfg = moe.make_config(16, 64, 8, 2, 128)
    n = moe.moe_workspace_bytes(cfg)
    c = ctypes.byref(cfg)
    inv, wsp = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_WORKSPACE
    f = P(FAKE)

    def back(dy=f, yp=f, inv_row=f, w=f, dyp=f, dw=f, ws=f, nb=n, cf=c):
        return lib.moe_combine_backward(cf, dy, yp, inv_row, w, dyp, dw, ws, nb, None)
    assert back(dyp=None, dw=None) == inv                     # nothing asked for
    assert back(dy=None) == inv and back(inv_row=None) == inv
    assert back(yp=None) == inv and back(w=None) == inv
    for name in ("dy", "yp", "dyp"):
        assert back(**{name: P(FAKE + 8)}) == inv
    for name in ("inv_row", "w", "dw"):
        assert back(**{name: P(FAKE + 2)}) == inv
    assert back(ws=None) == wsp and back(ws=P(FAKE + 8)) == wsp and back(nb=n - 1) == wsp
    assert back(cf=ctypes.byref(moe.make_config(16, 60, 8, 2, 128))) == inv


LINEAR = dict(M=16, n_in=64, n_out=33, act="gelu")
BAD_LINEAR = [dict(M=-1), dict(M=1 << 31), dict(n_in=0), dict(n_in=60), dict(n_out=0),
              dict(n_in=(1 << 20) + 8, ldx=1 << 21), dict(n_out=(1 << 20) + 1), dict(ldx=60),
              dict(ldx=68), dict(ldy=32), dict(ldr=32), dict(ldy=(1 << 32) + 8),
              dict(dtype="f32", n_in=62), dict(dtype="f32", out_dtype="bf16")]


@pytest.mark.parametrize("bad", BAD_LINEAR, ids=str)
def test_linear_config_refusals(lib, bad):
    good = moe.make_linear_config(**LINEAR)
    assert moe.moe_linear_workspace_bytes(good, True) >= moe.moe_linear_workspace_bytes(good, False) > 0
    cfg = moe.make_linear_config(**{**LINEAR, **bad})
    assert moe.moe_linear_workspace_bytes(cfg, False) == moe.moe_linear_workspace_bytes(cfg) == 0
    assert lib.moe_linear(ctypes.byref(cfg), *[P(FAKE)] * 7, 1 << 50, None) == moe.MOE_ERR_INVALID_ARG
    assert lib.moe_linear_backward(ctypes.byref(cfg), *[P(FAKE)] * 8, 1 << 50,
                                   None) == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("field,value", [("act", 5), ("act", -1), ("dtype", 2), ("out_dtype", 2)])
def test_linear_enum_refusals(lib, field, value):
    cfg = moe.make_linear_config(**LINEAR)
    setattr(cfg, field, value)
    assert moe.moe_linear_workspace_bytes(cfg) == 0


def test_linear_argument_refusals(lib):
    cfg = moe.make_linear_config(**LINEAR)
    c = ctypes.byref(cfg)
    inv, wsp = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_WORKSPACE
    f = P(FAKE)
    nf, nb_ = moe.moe_linear_workspace_bytes(cfg, False), moe.moe_linear_workspace_bytes(cfg, True)

    def fwd(x=f, W=f, b=f, r=f, y=f, z=f, ws=f, n=nf):
        return lib.moe_linear(c, x, W, b, r, y, z, ws, n, None)
    assert fwd(x=None) == inv and fwd(W=None) == inv and fwd(y=None) == inv
    assert fwd(x=P(FAKE + 8)) == inv and fwd(W=P(FAKE + 8)) == inv and fwd(b=P(FAKE + 2)) == inv
    assert fwd(r=P(FAKE + 1)) == inv and fwd(y=P(FAKE + 1)) == inv and fwd(z=P(FAKE + 1)) == inv
    assert fwd(ws=None) == wsp and fwd(ws=P(FAKE + 8)) == wsp and fwd(n=nf - 1) == wsp

    def back(dy=f, x=f, W=f, z=f, dx=f, dW=f, db=f, ws=f, n=nb_):
        return lib.moe_linear_backward(c, dy, x, W, z, dx, dW, db, ws, n, None)
    assert back(dx=None, dW=None, db=None) == inv
    for name in ("dy", "x", "W", "z"):
        assert back(**{name: None}) == inv
    for name in ("x", "W", "dx", "dW"):
        assert back(**{name: P(FAKE + 8)}) == inv
    assert back(dy=P(FAKE + 1)) == inv and back(z=P(FAKE + 1)) == inv and back(db=P(FAKE + 2)) == inv
    assert back(ws=None) == wsp and back(ws=P(FAKE + 8)) == wsp and back(n=nb_ - 1) == wsp


class OnDevice:
    """A host tensor that answers as one on cuda:0 would: the binding's own checks come before
    anything is launched, so they can be seen without a GPU."""

    def __init__(self, t, index=0):
        self._t, self._index = t, index

    def __getattr__(self, name):
        return getattr(self._t, name)

    is_cuda = True

    def get_device(self):
        return self._index


def test_binding_refuses_wrong_tensors(lib):
    """Element type, shape, strides and device are checked where the C call sees addresses only."""
    cfg = moe.make_route_config(4, 8, 2)
    ws = OnDevice(torch.zeros(moe.moe_route_workspace_bytes(cfg), dtype=torch.uint8))
    l, idx, w = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    bad = [(l.double(), None, idx, w), (l[:3], None, idx, w), (torch.zeros(8, 4).t(), None, idx, w),
           (torch.zeros(4, 16)[:, ::2], None, idx, w), (torch.zeros(4, 9)[:, :8], None, idx, w),
           (l, torch.zeros(7), idx, w), (l, None, idx.long(), w), (l, None, idx, w.half()),
           (l, None, torch.zeros(2, 4, dtype=torch.int32).t(), w), (None, None, idx, w),
           (l, None, None, w)]
    for args in bad:
        with pytest.raises(moe.MoeError) as err:
            moe.moe_route(cfg, *[None if a is None else OnDevice(a) for a in args], None, ws)
        assert err.value.status == moe.MOE_ERR_INVALID_ARG
    with pytest.raises(moe.MoeError) as err:                  # on another device than the workspace
        moe.moe_route(cfg, OnDevice(l, 1), None, OnDevice(idx), OnDevice(w), None, ws)
    assert err.value.status == moe.MOE_ERR_INVALID_ARG
    for other in (ws._t, OnDevice(ws._t[::2])):               # a workspace on the host, or with gaps
        with pytest.raises(moe.MoeError) as err:
            moe.moe_route(cfg, OnDevice(l), None, OnDevice(idx), OnDevice(w), None, other)
        assert err.value.status == moe.MOE_ERR_WORKSPACE
    padded = moe.make_route_config(4, 8, 2, ld=9)
    with pytest.raises(moe.MoeError):                         # gaps announced, but not there
        moe.moe_route(padded, OnDevice(l), None, OnDevice(idx), OnDevice(w), None, ws)
    lc = moe.make_linear_config(4, 8, 3)
    x, W, y = torch.zeros(4, 8).bfloat16(), torch.zeros(3, 8).bfloat16(), torch.zeros(4, 3).bfloat16()
    for args in ((x.float(), W, y), (x, W.t().contiguous(), y), (x, W, y.float())):
        a = [OnDevice(t) for t in args]
        with pytest.raises(moe.MoeError):
            moe.moe_linear(lc, a[0], a[1], None, None, a[2], None, ws)
    with pytest.raises(moe.MoeError):
        moe.route_workspace(moe.make_route_config(4, 8, 9))
    with pytest.raises(moe.MoeError):
        moe.linear_workspace(moe.make_linear_config(4, 7, 9))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_definition_against_differences(score, renorm):
    rng = np.random.default_rng(3)
    T, N, k = 3, 7, 3
    l = rng.normal(size=(T, N))
    idx, _, _ = gate_ref.route(l, rng.normal(size=N) * 0.1, k, score)
    g, c = rng.normal(size=(T, k)), rng.normal(size=N) * T
    grad, _ = gate_ref.route_grad(l, idx, g, c, score, renorm, 2.5)
    h = 1e-6
    for t in range(T):
        for e in range(N):
            d = np.zeros_like(l)
            d[t, e] = h
            num = (gate_ref.route_loss(l + d, idx, g, c, score, renorm, 2.5) -
                   gate_ref.route_loss(l - d, idx, g, c, score, renorm, 2.5)) / (2 * h)
            # the difference's own error: h^2 f''' / 6 and 2 ulp(L) / h, both under 1e-8
            assert abs(num - grad[t, e]) < 1e-8


@pytest.mark.parametrize("name", ["none", "relu", "silu", "gelu", "gelu_tanh"])
def test_activation_gradient_definition_against_differences(name):
    z = np.linspace(-6, 6, 101) + 0.013       # not at relu's corner
    h = 1e-6
    num = (gate_ref.act(name, z + h) - gate_ref.act(name, z - h)) / (2 * h)
    assert np.abs(num - gate_ref.act_grad(name, z)).max() < 1e-8
