"""One buffer as the workspace of several configurations: the words that have to be zero between
calls lie in the same head of every workspace, and all behind the head is written before it is read."""
import ctypes
import os
import re

import pytest
import torch

import synth
import top_routing_expert_warp_b200 as moe
from gpu_util import LayerRun, upload_inputs
from top_routing_expert_warp_b200 import build as moe_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TD = {"f32": torch.float32, "bf16": torch.bfloat16}
HEAD = 4352          # the status word's 256 bytes and two arrays of 512 counters


def test_every_workspace_begins_with_the_same_head():
    moe_build.build()
    txt = open(os.path.join(ROOT, "include", "moe.h")).read()
    assert int(re.search(r"MOE_WORKSPACE_HEAD = (\d+)", txt).group(1)) == moe.MOE_WORKSPACE_HEAD == HEAD
    for dtype in ("f32", "bf16"):
        for M in (0, 1, 200, 333):
            cfg = moe.make_linear_config(M, 16, 12, dtype=dtype)
            assert moe.moe_linear_workspace_bytes(cfg, False) >= HEAD
            assert moe.moe_linear_workspace_bytes(cfg, True) >= HEAD
    # routing: the blocks' sums (at most 592 blocks of N doubles) behind the head
    assert moe.moe_route_workspace_bytes(moe.make_route_config(4, 32, 2)) >= HEAD + 592 * 32 * 8
    # the layer: its first region is the router's sums, then (fp32) the chosen experts
    one = moe.moe_workspace_layout(moe.make_config(4, 64, 8, 2, 16, dtype="f32"))["topk_idx"]
    two = moe.moe_workspace_layout(moe.make_config(4, 64, 16, 2, 16, dtype="f32"))["topk_idx"]
    assert one - (two - one) == HEAD             # the sums' size goes with the experts alone


def grads(cfg, ws, dt, seed):
    """dx, dW and db of one projection, outputs filled with a mark first."""
    g = torch.Generator().manual_seed(seed)
    M, K, N = cfg.M, cfg.n_in, cfg.n_out
    x, W, dy = (torch.randn(*s, generator=g).to(TD[dt]).cuda() for s in ((M, K), (N, K), (M, N)))
    y = torch.full((M, N), 7.0, dtype=TD[dt], device="cuda")
    out = [torch.full_like(x, 7.0), torch.full_like(W, 7.0), torch.full((N,), 7.0, device="cuda")]
    moe.moe_linear(cfg, x, W, None, None, y, None, ws)
    moe.moe_linear_backward(cfg, dy, x, W, None, *out, ws)
    assert moe.moe_check_status(ws)[0] == moe.MOE_OK
    return [y] + out


@pytest.mark.gpu
def test_projections_of_changing_sizes_and_types_share_a_workspace():
    """A last batch that is shorter, other widths and the other type on one buffer: the results are
    those of workspaces of their own, bit for bit."""
    calls = [("f32", 333, 516, 129), ("f32", 200, 516, 129), ("bf16", 333, 520, 136), ("f32", 333, 516, 129),
             ("f32", 64, 1024, 64), ("bf16", 1000, 264, 512), ("f32", 200, 516, 129), ("f32", 64, 1024, 64)]
    cfgs = [moe.make_linear_config(M, K, N, dtype=dt) for dt, M, K, N in calls]
    shared = torch.zeros(max(moe.moe_linear_workspace_bytes(c) for c in cfgs), dtype=torch.uint8, device="cuda")
    for i, (cfg, (dt, *_)) in enumerate(zip(cfgs, calls)):
        want = grads(cfg, moe.linear_workspace(cfg), dt, i)
        got = grads(cfg, shared, dt, i)
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_the_gate_the_layer_and_a_projection_share_a_workspace():
    T, d, N, k, H = 200, 256, 8, 2, 128
    lc = moe.make_linear_config(T, d, N, dtype="f32")
    rc = moe.make_route_config(T, N, k, renormalize=True)
    cfg = moe.make_config(T, d, N, k, H, dtype="f32")
    shared = torch.zeros(max(moe.moe_linear_workspace_bytes(lc), moe.moe_route_workspace_bytes(rc),
                             moe.moe_workspace_bytes(cfg)), dtype=torch.uint8, device="cuda")
    g = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    x, Wg, dy, dyl = rnd(T, d), rnd(N, d) * d ** -0.5, rnd(T, d), rnd(T, N)
    W1, W3, W2 = rnd(N, H, d) * d ** -0.5, rnd(N, H, d) * d ** -0.5, rnd(N, d, H) * H ** -0.5
    e = lambda *s, dtype=torch.float32: torch.full(s, 7, dtype=dtype, device="cuda")  # noqa: E731
    i32 = torch.int32

    def step(lws, rws, ws):
        l, idx, w, p, y = e(T, N), e(T, k, dtype=i32), e(T, k), e(N), e(T, d)
        moe.moe_linear(lc, x, Wg, None, None, l, None, lws)
        moe.moe_route(rc, l, None, idx, w, p, rws)
        R = T * k
        counts, offs, perm, inv = e(N, dtype=i32), e(N + 1, dtype=i32), e(R, dtype=i32), e(R, dtype=i32)
        drop, xp, yp = e(R, dtype=torch.uint8), e(R, d), e(R, d)
        moe.moe_dispatch(cfg, x, idx, counts, offs, perm, inv, drop, xp, None, p, e(N), e(1), ws)
        moe.moe_expert_ffn(cfg, xp, None, offs, W1, W3, W2, yp, ws)
        moe.moe_combine(cfg, yp, inv, w, None, y, ws)
        dyp, dw, dl, dx, dW = e(R, d), e(T, k), e(T, N), e(T, d), e(N, d)
        moe.moe_combine_backward(cfg, dy, yp, inv, w, dyp, dw, ws)
        moe.moe_route_backward(rc, l, idx, dw, p, dl, rws)
        moe.moe_linear_backward(lc, dl + dyl, x, Wg, None, dx, dW, None, lws)
        return [l, idx, w, p, y, dyp, dw, dl, dx, dW]
    want = step(moe.linear_workspace(lc), moe.route_workspace(rc), moe.workspace(cfg))
    for _ in range(2):
        for a, b in zip(step(shared, shared, shared), want):
            assert torch.equal(a, b)
    assert moe.moe_check_status(shared)[0] == moe.MOE_OK


@pytest.mark.gpu
def test_captured_graphs_of_two_sizes_share_a_workspace():
    calls = [(333, 516, 129), (200, 516, 129)]
    cfgs = [moe.make_linear_config(*c, dtype="f32") for c in calls]
    shared = torch.zeros(max(moe.moe_linear_workspace_bytes(c) for c in cfgs), dtype=torch.uint8, device="cuda")
    want = [grads(c, moe.linear_workspace(c), "f32", i)[1:] for i, c in enumerate(cfgs)]
    graphs = []
    for i, (M, K, N) in enumerate(calls):
        gen = torch.Generator().manual_seed(i)
        x, W, dy = (torch.randn(*s, generator=gen).cuda() for s in ((M, K), (N, K), (M, N)))
        out = [torch.zeros_like(x), torch.zeros_like(W), torch.zeros(N, device="cuda")]
        moe.moe_linear_backward(cfgs[i], dy, x, W, None, *out, shared)      # first use outside the capture
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.moe_linear_backward(cfgs[i], dy, x, W, None, *out, shared)
        graphs.append((graph, out, (x, W, dy)))
    for i in (0, 1, 0, 1, 1, 0):
        graph, out, _ = graphs[i]
        for t in out:
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want[i]):
            assert torch.equal(a, b)


LAYERS = {
    "fp32": synth.TINY_F32,
    "fp32-capacity": synth.TINY_F32.with_(capacity_factor=0.6, seed=41),
    "top2": synth.MIXTRAL.with_(T=300, d=256, H=384),
    "drops": synth.SWITCH.with_(T=1000, d=128, H=256),
    "fallback": synth.SWITCH.with_(T=700, d=128, H=256, overflow="fallback", capacity_factor=0.5, seed=42),
    "fp8-shared": synth.DEEPSEEK.with_(T=200, d=256, H=128, H_shared=128),
    "fp8": synth.DEEPSEEK.with_(T=300, d=272, H=192, H_shared=0, seed=31),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(LAYERS))
def test_layers_do_not_read_what_others_left(name):
    """Any bytes behind the head (NaN patterns among them) change nothing."""
    wl = LAYERS[name]
    dev, _ = upload_inputs(wl)
    run = LayerRun(wl, dev)
    outs = lambda: [t.clone() for t in (run(), run.topk_idx, run.topk_w, run.counts, run.f,  # noqa: E731
                                        run.p_mean, run.aux)]
    want = outs()
    g = torch.Generator(device="cuda").manual_seed(3)
    for fill in (None, 255, 127):
        if fill is None:
            run.ws[HEAD:].random_(0, 256, generator=g)
        else:
            run.ws[HEAD:] = fill
        for a, b in zip(outs(), want):
            assert torch.equal(a, b)
    assert run.check_status()[0] == moe.MOE_OK


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_the_gate_and_projections_do_not_read_what_others_left(dt):
    cfg = moe.make_linear_config(300, 1032, 137, dtype=dt)
    ws = moe.linear_workspace(cfg)
    want = grads(cfg, ws, dt, 5)
    rc = moe.make_route_config(5000, 96, 4, score="sigmoid")
    l = torch.randn(5000, 96, generator=torch.Generator().manual_seed(2)).cuda()

    def route(w):
        idx, tw = torch.empty(5000, 4, dtype=torch.int32, device="cuda"), torch.empty(5000, 4, device="cuda")
        p = torch.empty(96, device="cuda")
        moe.moe_route(rc, l, None, idx, tw, p, w)
        return [idx, tw, p]
    rws = moe.route_workspace(rc)
    want_r = route(rws)
    for fill in (255, 127):
        ws[HEAD:] = fill
        rws[HEAD:] = fill
        for a, b in zip(grads(cfg, ws, dt, 5) + route(rws), want + want_r):
            assert torch.equal(a, b)


def test_a_workspace_without_room_for_the_head_is_refused():
    moe_build.build()
    lib = moe.lib()
    p = ctypes.c_void_p(1 << 40)                 # never dereferenced: validation fails first
    lc = moe.make_linear_config(4, 16, 8)
    assert lib.moe_linear(ctypes.byref(lc), p, p, None, None, p, None, p, HEAD - 1, None) == moe.MOE_ERR_WORKSPACE
    rc = moe.make_route_config(4, 16, 2)
    assert lib.moe_route(ctypes.byref(rc), p, None, p, p, None, p, HEAD - 1, None) == moe.MOE_ERR_WORKSPACE
