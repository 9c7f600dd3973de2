"""Measured cases of the trainable gate and the dense projections around the experts.

Routing of given logits to experts (``moe_route``) and its gradient
(``moe_route_backward``), the gradient of the gate-weighted combine
(``moe_combine_backward``), and the dense projection with bias, activation and
residual (``moe_linear``) and its gradients (``moe_linear_backward``).  With
``own`` false every case runs in its plain form, elementary torch operations;
with ``own`` true it runs through the package.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
def listed():
    deepseek = dict(score="sigmoid", N=256, k=8, n_groups=8, topk_groups=4, group_top=2, bias=True,
                    renormalize=True, scale=2.5)
    return [
        # one token of a serving step through a 256-expert gate: latency
        dict(name="route_one_token", op="route", T=1, dtype="f32", pad=0, dead=0, **deepseek),
        # the same gate over the tokens of a prompt batch, with the balance statistics
        dict(name="route_prompt", op="route", T=4096, dtype="f32", pad=0, dead=0, **deepseek),
        # a top-1 softmax gate on a long bf16 batch; the logits are columns of a wider
        # buffer and three experts are switched off (-inf)
        dict(name="route_top1_bf16", op="route", T=32771, dtype="bf16", pad=8, dead=3,
             score="softmax", N=128, k=1, n_groups=0, topk_groups=0, group_top=0, bias=False,
             renormalize=False, scale=1.0),
        # training step of the 256-expert gate on a large batch
        dict(name="route_grad_large", op="route_grad", T=65536, dtype="f32", pad=0, **deepseek),
        # training step of a small odd softmax gate in bf16
        dict(name="route_grad_odd", op="route_grad", T=1003, dtype="bf16", pad=4, score="softmax",
             N=60, k=4, n_groups=0, topk_groups=0, group_top=0, bias=False, renormalize=True,
             scale=1.0),
        # combine's gradient for 4096 tokens of an 8-expert top-2 layer
        dict(name="combine_grad_top2", op="combine_grad", T=4096, d=4096, N=8, k=2, dtype="bf16",
             cf=0.0),
        # many small shares per token, with capacity dropping
        dict(name="combine_grad_drops", op="combine_grad", T=4099, d=2048, N=256, k=8,
             dtype="bf16", cf=8.0),
        # one decode token through a dense up-projection: the weights' bytes
        dict(name="linear_one_token", op="linear", M=1, n_in=7168, n_out=2048, act="silu",
             dtype="bf16", out="bf16", bias=True, residual=False, preact=False, pad=0),
        # router projection of a prompt batch to fp32 logits
        dict(name="linear_router", op="linear", M=4096, n_in=7168, n_out=256, act="none",
             dtype="bf16", out="f32", bias=False, residual=False, preact=False, pad=0),
        # dense down-projection with the block's residual, training batch
        dict(name="linear_large", op="linear", M=4096, n_in=4096, n_out=14336, act="gelu",
             dtype="bf16", out="bf16", bias=True, residual=True, preact=True, pad=0),
        # gradients of a dense projection, training batch
        dict(name="linear_grad_large", op="linear_grad", M=4096, n_in=4096, n_out=4096,
             act="gelu", dtype="bf16", out="bf16", bias=True, pad=0),
        # gradients of a small odd fp32 projection, strided rows
        dict(name="linear_grad_f32", op="linear_grad", M=333, n_in=516, n_out=129, act="silu",
             dtype="f32", out="f32", bias=True, pad=4),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_gate(rng):
    N = rng.choice([rng.randint(1, 256), 64, 128, 160, 256])
    k = rng.randint(1, min(8, N))
    n_groups = topk_groups = group_top = 0
    ways = [g for g in (2, 4, 8, 16) if N % g == 0 and N // g >= 2]
    if ways and rng.random() < 0.5:
        n_groups = rng.choice(ways)
        per = N // n_groups
        low = -(-k // per)
        if low < n_groups:
            topk_groups = rng.randint(low, n_groups - 1)
            group_top = rng.randint(1, min(per, 3))
        else:
            n_groups = 0
    return dict(score=rng.choice(["sigmoid", "softmax"]), N=N, k=k, n_groups=n_groups,
                topk_groups=topk_groups, group_top=group_top, bias=rng.random() < 0.5,
                renormalize=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]))


def draw(rng):
    op = rng.choice(["route", "route_grad", "combine_grad", "linear", "linear_grad"])
    if op in ("route", "route_grad"):
        c = dict(op=op, T=_log_int(rng, 1, 32768), dtype=rng.choice(["f32", "bf16"]),
                 pad=rng.choice([0, 0, 1, 8]), **_draw_gate(rng))
        if op == "route":
            c["dead"] = rng.choice([0, 0, 1]) if c["N"] - c["k"] > 0 and c["n_groups"] == 0 else 0
        return c
    if op == "combine_grad":
        f32 = rng.random() < 0.3
        N = rng.randint(1, 16) if f32 else rng.choice([8, 64, 128, 256, rng.randint(1, 256)])
        k = rng.randint(1, min(8, N))
        d = 8 * _log_int(rng, 8, 512)
        T = _log_int(rng, 1, max(2, (1 << 25) // (d * k)))
        return dict(op=op, T=T, d=d, N=N, k=k, dtype="f32" if f32 else "bf16",
                    cf=rng.choice([0.0, 0.75 * k, 1.25 * k]))
    dtype = rng.choice(["bf16", "bf16", "f32"])
    top = 4096 if dtype == "bf16" else 1024
    c = dict(op=op, M=_log_int(rng, 1, top), n_in=8 * _log_int(rng, 4, top // 8),
             n_out=_log_int(rng, 1, top), act=rng.choice(ACTS), dtype=dtype,
             out=rng.choice([dtype, "f32"]), bias=rng.random() < 0.7, pad=rng.choice([0, 0, 8]))
    if op == "linear":
        c["residual"] = rng.random() < 0.5
        c["preact"] = rng.random() < 0.3
    return c


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 13)
    return g


def _randn(g, *shape, std=1.0, dtype=torch.float32):
    out = torch.empty(shape, dtype=torch.float32, device="cuda")
    out.normal_(0.0, std, generator=g)
    return out.to(dtype)


def _strided(t, pad):
    """The rows of t as columns of a buffer that is `pad` wider."""
    if not pad:
        return t
    wide = torch.zeros(t.shape[0], t.shape[1] + pad, dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def _gate_inputs(case, g):
    T, N, k = case["T"], case["N"], case["k"]
    logits = _randn(g, T, N, std=1.5, dtype=DTYPE[case["dtype"]])
    if case.get("dead"):
        off = torch.randperm(N, generator=g, device="cuda")[:case["dead"]]
        logits[:, off] = float("-inf")
    bias = _randn(g, N, std=0.05) if case["bias"] else None
    return _strided(logits, case["pad"]), bias


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=case)
    op = case["op"]
    if op in ("route", "route_grad"):
        st["logits"], st["bias"] = _gate_inputs(case, g)
        T, N, k = case["T"], case["N"], case["k"]
        if op == "route_grad":
            l64 = st["logits"].double()
            st["topk_idx"] = _choose(case, l64, _scores(case, l64), st["bias"]).to(torch.int32)
            st["dtopk_w"] = _randn(g, T, k, std=0.1)
            st["dp_mean"] = _randn(g, N, std=0.05 * T)
    elif op == "combine_grad":
        T, d, N, k = case["T"], case["d"], case["N"], case["k"]
        dt = DTYPE[case["dtype"]]
        idx = torch.rand(T, N, device="cuda", generator=g).argsort(dim=1)[:, :k]
        order = idx.reshape(-1).argsort(stable=True)
        e = idx.reshape(-1)[order]
        first = torch.searchsorted(e, torch.arange(N, device="cuda"))
        within = torch.arange(T * k, device="cuda") - first[e]
        cap = int(case["cf"] * T / N) if case["cf"] > 0 else T * k
        keep = within < cap
        row = torch.where(keep, keep.long().cumsum(0) - 1, torch.full_like(within, -1))
        inv = torch.empty(T * k, dtype=torch.int32, device="cuda")
        inv[order] = row.to(torch.int32)
        st["inv_row"] = inv
        st["topk_w"] = torch.rand(T, k, device="cuda", generator=g)
        st["dy"] = _randn(g, T, d, dtype=dt)
        st["y_perm"] = _randn(g, T * k, d, dtype=dt)
    else:
        M, K, N = case["M"], case["n_in"], case["n_out"]
        dt, od = DTYPE[case["dtype"]], DTYPE[case["out"]]
        st["x"] = _strided(_randn(g, M, K, dtype=dt), case["pad"])
        st["W"] = _randn(g, N, K, std=K ** -0.5, dtype=dt)
        st["bias"] = _randn(g, N, std=0.1) if case["bias"] else None
        if op == "linear":
            st["residual"] = _strided(_randn(g, M, N, dtype=od), case["pad"]) if case["residual"] else None
        else:
            st["dy"] = _strided(_randn(g, M, N, dtype=od), case["pad"])
            st["preact"] = _randn(g, M, N, dtype=dt) if case["act"] != "none" else None
    if own:
        _prepare_own(case, st)
    return st


def _prepare_own(case, st):
    import top_routing_expert_warp_b200 as moe
    op = case["op"]
    empty = lambda *s, dtype: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    if op in ("route", "route_grad"):
        T, N, k = case["T"], case["N"], case["k"]
        st["cfg"] = moe.make_route_config(T, N, k, score=case["score"], n_groups=case["n_groups"],
                                          topk_groups=case["topk_groups"], group_top=case["group_top"],
                                          renormalize=case["renormalize"], scale=case["scale"],
                                          dtype=case["dtype"], ld=N + case["pad"])
        st["ws"] = moe.route_workspace(st["cfg"])
        if op == "route":
            st["topk_idx"] = empty(T, k, dtype=torch.int32)
            st["topk_w"] = empty(T, k, dtype=torch.float32)
            st["p_mean"] = empty(N, dtype=torch.float32)
        else:
            st["dlogits"] = _strided(empty(T, N, dtype=DTYPE[case["dtype"]]), case["pad"])
    elif op == "combine_grad":
        T, d, N, k = case["T"], case["d"], case["N"], case["k"]
        st["cfg"] = moe.make_config(T, d, N, k, 8, dtype=case["dtype"], capacity_factor=case["cf"])
        st["ws"] = moe.workspace(st["cfg"])
        # rows behind the last kept one are left as they are
        st["dy_perm"] = torch.zeros(T * k, d, dtype=DTYPE[case["dtype"]], device="cuda")
        st["dtopk_w"] = empty(T, k, dtype=torch.float32)
    else:
        M, K, N, pad = case["M"], case["n_in"], case["n_out"], case["pad"]
        dt, od = DTYPE[case["dtype"]], DTYPE[case["out"]]
        st["cfg"] = moe.make_linear_config(M, K, N, act=case["act"], dtype=case["dtype"],
                                           out_dtype=case["out"], ldx=K + pad, ldy=N + pad, ldr=N + pad)
        st["ws"] = moe.linear_workspace(st["cfg"])
        if op == "linear":
            st["y"] = _strided(empty(M, N, dtype=od), pad)
            st["z"] = empty(M, N, dtype=dt) if case["preact"] else None
        else:
            st["dx"] = _strided(empty(M, K, dtype=dt), pad)
            st["dW"] = empty(N, K, dtype=dt)
            st["db"] = empty(N, dtype=torch.float32) if case["bias"] else None


# ------------------------------------------------------------------ plain forms
def _scores(case, l64):
    """Scores in 64 bits: the choice of experts hangs on differences between them."""
    if case["score"] == "sigmoid":
        return torch.sigmoid(l64)
    top = l64.amax(dim=1, keepdim=True)
    e = torch.exp(l64 - top)
    return e / e.sum(dim=1, keepdim=True)


def _choose(case, l64, s, bias):
    T, N = l64.shape
    off = l64 == float("-inf")
    v = l64 if bias is None else (s + bias.double()).masked_fill(off, float("-inf"))
    if case["n_groups"] > 1 and case["topk_groups"] < case["n_groups"]:
        G, per = case["n_groups"], N // case["n_groups"]
        sv = s if bias is None else s + bias.double()
        sv = sv.masked_fill(off, float("-inf")).view(T, G, per)
        best = torch.sort(sv, dim=2, descending=True, stable=True).values[:, :, :case["group_top"]]
        gs = best.masked_fill(best == float("-inf"), 0.0).sum(dim=2)
        gi = torch.sort(gs, dim=1, descending=True, stable=True).indices[:, :case["topk_groups"]]
        allowed = torch.zeros(T, G, dtype=torch.bool, device=v.device).scatter_(1, gi, True)
        v = v.masked_fill(~allowed.repeat_interleave(per, dim=1), float("-inf"))
    return torch.sort(v, dim=1, descending=True, stable=True).indices[:, :case["k"]]


def _plain_route(st):
    case = st["case"]
    l64 = st["logits"].double()
    s = _scores(case, l64)
    idx = _choose(case, l64, s, st["bias"])
    w = torch.gather(s, 1, idx)
    if case["renormalize"]:
        w = w / w.sum(dim=1, keepdim=True)
    p = (s / s.sum(dim=1, keepdim=True)).mean(dim=0)
    return idx.to(torch.int32), (w * case["scale"]).float(), p.float()


def _plain_route_grad(st):
    case = st["case"]
    l = st["logits"].float()
    idx, g = st["topk_idx"].long(), st["dtopk_w"] * case["scale"]
    c = st["dp_mean"] / case["T"]
    if case["score"] == "sigmoid":
        s = torch.sigmoid(l)
        one_minus = torch.sigmoid(-l)
    else:
        e = torch.exp(l - l.amax(dim=1, keepdim=True))
        s = e / e.sum(dim=1, keepdim=True)
    sk = torch.gather(s, 1, idx)
    if case["renormalize"]:
        D = sk.sum(dim=1, keepdim=True)
        gs = (g - (g * sk).sum(dim=1, keepdim=True) / D) / D
    else:
        gs = g
    ds = torch.zeros_like(s).scatter_(1, idx, gs)
    Z = s.sum(dim=1, keepdim=True)
    ds = ds + (c - (c * s).sum(dim=1, keepdim=True) / Z) / Z
    if case["score"] == "sigmoid":
        dl = s * one_minus * ds
    else:
        dl = s * (ds - (s * ds).sum(dim=1, keepdim=True))
    return dl.to(st["logits"].dtype)


def _plain_combine_grad(st):
    case = st["case"]
    T, d, k = case["T"], case["d"], case["k"]
    dy = st["dy"].float()
    inv = st["inv_row"].view(T, k).long()
    kept = inv >= 0
    rows = torch.where(kept, inv, torch.full_like(inv, T * k))      # dropped: a row behind the others
    out = torch.zeros(T * k + 1, d, dtype=st["dy"].dtype, device=dy.device)
    dw = []
    for j in range(k):
        y = st["y_perm"][inv[:, j].clamp(min=0)].float()
        dw.append((dy * y).sum(dim=1) * kept[:, j])
        out[rows[:, j]] = (st["topk_w"][:, j:j + 1] * dy).to(out.dtype)
    return out[:T * k], torch.stack(dw, dim=1)


def _act(name, z):
    if name == "relu":
        return torch.clamp(z, min=0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
    return z


def _act_grad(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    if name == "gelu_tanh":
        a = (2 / math.pi) ** 0.5
        t = torch.tanh(a * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _plain_linear(st):
    case = st["case"]
    z = st["x"].float() @ st["W"].float().t()
    if st["bias"] is not None:
        z = z + st["bias"]
    y = _act(case["act"], z)
    if st["residual"] is not None:
        y = y + st["residual"].float()
    y = y.to(DTYPE[case["out"]])
    return (y, z.to(DTYPE[case["dtype"]])) if case["preact"] else (y,)


def _plain_linear_grad(st):
    case = st["case"]
    dt = DTYPE[case["dtype"]]
    dz = st["dy"].float()
    if case["act"] != "none":
        dz = dz * _act_grad(case["act"], st["preact"].float())
    dx = (dz @ st["W"].float()).to(dt)
    dW = (dz.t() @ st["x"].float()).to(dt)
    return (dx, dW, dz.sum(dim=0)) if case["bias"] else (dx, dW)


PLAIN = dict(route=_plain_route, route_grad=_plain_route_grad, combine_grad=_plain_combine_grad,
             linear=_plain_linear, linear_grad=_plain_linear_grad)


def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return PLAIN[op](st)
    import top_routing_expert_warp_b200 as moe
    if op == "route":
        moe.moe_route(st["cfg"], st["logits"], st["bias"], st["topk_idx"], st["topk_w"],
                      st["p_mean"], st["ws"])
        return st["topk_idx"], st["topk_w"], st["p_mean"]
    if op == "route_grad":
        moe.moe_route_backward(st["cfg"], st["logits"], st["topk_idx"], st["dtopk_w"],
                               st["dp_mean"], st["dlogits"], st["ws"])
        return st["dlogits"]
    if op == "combine_grad":
        moe.moe_combine_backward(st["cfg"], st["dy"], st["y_perm"], st["inv_row"], st["topk_w"],
                                 st["dy_perm"], st["dtopk_w"], st["ws"])
        return st["dy_perm"], st["dtopk_w"]
    if op == "linear":
        moe.moe_linear(st["cfg"], st["x"], st["W"], st["bias"], st["residual"], st["y"], st["z"],
                       st["ws"])
        return (st["y"], st["z"]) if case["preact"] else (st["y"],)
    moe.moe_linear_backward(st["cfg"], st["dy"], st["x"], st["W"], st["preact"], st["dx"],
                            st["dW"], st["db"], st["ws"])
    return (st["dx"], st["dW"], st["db"]) if case["bias"] else (st["dx"], st["dW"])


# ------------------------------------------------------------------ work of one pass
def work(case):
    op = case["op"]
    es = {"f32": 4, "bf16": 2}
    if op in ("route", "route_grad"):
        T, N, k = case["T"], case["N"], case["k"]
        e = es[case["dtype"]]
        if op == "route":
            return dict(bytes=T * N * e + T * k * 8 + N * 4 * (2 if case["bias"] else 1),
                        flops=T * N * 6)
        return dict(bytes=2 * T * N * e + T * k * 8 + N * 4, flops=T * N * 10)
    if op == "combine_grad":
        T, d, N, k = case["T"], case["d"], case["N"], case["k"]
        e = es[case["dtype"]]
        # rows kept when the experts are chosen evenly: all of them, or the capacity
        R = T * k if case["cf"] <= 0 else min(T * k, N * int(case["cf"] * T / N))
        return dict(bytes=(T * d + 2 * R * d) * e + T * k * 12, flops=3 * R * d)
    M, K, N = case["M"], case["n_in"], case["n_out"]
    e, o = es[case["dtype"]], es[case["out"]]
    if op == "linear":
        b = (M * K + N * K) * e + M * N * o * (2 if case["residual"] else 1)
        b += (M * N * e if case["preact"] else 0) + (4 * N if case["bias"] else 0)
        return dict(bytes=b, flops=2 * M * N * K)
    b = M * N * o + (M * N * e if case["act"] != "none" else 0) + 2 * (M * K + N * K) * e
    return dict(bytes=b + (4 * N if case["bias"] else 0), flops=4 * M * N * K)


# ------------------------------------------------------------------ definitions in 64 bits
def _exact_route(case, st):
    """Token by token from the definition, on the host."""
    import numpy as np
    l = st["logits"].double().cpu().numpy()
    b = st["bias"].double().cpu().numpy() if st["bias"] is not None else None
    T, N = l.shape
    k = case["k"]
    dead = np.isneginf(l)
    if case["score"] == "sigmoid":
        with np.errstate(over="ignore"):
            s = 1.0 / (1.0 + np.exp(-l))
    else:
        s = np.exp(l - l.max(1, keepdims=True))
        s /= s.sum(1, keepdims=True)
    rank = l if b is None else np.where(dead, -np.inf, s + b)
    if case["n_groups"] > 1 and case["topk_groups"] < case["n_groups"]:
        G = case["n_groups"]
        val = np.where(dead, -np.inf, s if b is None else s + b).reshape(T, G, N // G)
        val = -np.sort(-val, axis=2)[:, :, :case["group_top"]]
        score = np.where(np.isneginf(val), 0.0, val).sum(2)
        order = np.argsort(-score, axis=1, kind="stable")[:, :case["topk_groups"]]
        node = np.zeros((T, G), bool)
        np.put_along_axis(node, order, True, axis=1)
        rank = np.where(np.repeat(node, N // G, axis=1), rank, -np.inf)
    idx = np.argsort(-rank, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(s, idx, axis=1)
    if case["renormalize"]:
        w = w / w.sum(1, keepdims=True)
    p = (s / s.sum(1, keepdims=True)).mean(0)
    return (torch.from_numpy(idx.astype(np.int32)), torch.from_numpy(w * case["scale"]),
            torch.from_numpy(p))


def _exact_grad(outs, grads, leaves):
    """Vector-Jacobian product by automatic differentiation of the forward definition."""
    total = sum((o * g).sum() for o, g in zip(outs, grads))
    return torch.autograd.grad(total, leaves)


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = kept
    op = case["op"]
    if op == "route":
        return _exact_route(case, st)
    if op == "route_grad":
        parts = []
        for t in range(0, case["T"], 8192):
            l = st["logits"][t:t + 8192].double().requires_grad_(True)
            s = torch.softmax(l, 1) if case["score"] == "softmax" else 1 / (1 + torch.exp(-l))
            w = s.gather(1, st["topk_idx"][t:t + 8192].long())
            if case["renormalize"]:
                w = w / w.sum(1, keepdim=True)
            p = (s / s.sum(1, keepdim=True)).sum(0) / case["T"]
            parts += _exact_grad([w * case["scale"], p],
                                 [st["dtopk_w"][t:t + 8192].double(), st["dp_mean"].double()], [l])
        return torch.cat(parts)
    if op == "combine_grad":
        T, d, k = case["T"], case["d"], case["k"]
        inv = st["inv_row"].long()
        pair = torch.nonzero(inv >= 0).flatten()
        row, tok = inv[pair], pair // k
        out = torch.zeros(T * k, d, dtype=torch.float64, device="cuda")
        dw = torch.zeros(T * k, dtype=torch.float64, device="cuda")
        w = st["topk_w"].flatten().double()
        for a in range(0, len(pair), 8192):
            r, t, q = row[a:a + 8192], tok[a:a + 8192], pair[a:a + 8192]
            g = st["dy"][t].double()
            out[r] = w[q, None] * g
            dw[q] = torch.einsum("rd,rd->r", g, st["y_perm"][r].double())
        return out, dw.view(T, k)
    x, W = st["x"].double(), st["W"].double()
    fn = dict(none=lambda z: z, relu=torch.relu, silu=torch.nn.functional.silu,
              gelu=torch.nn.functional.gelu,
              gelu_tanh=lambda z: torch.nn.functional.gelu(z, approximate="tanh"))[case["act"]]
    if op == "linear":
        z = torch.einsum("mk,nk->mn", x, W)
        if st["bias"] is not None:
            z = z + st["bias"].double()
        y = fn(z)
        if st["residual"] is not None:
            y = y + st["residual"].double()
        return (y, z) if case["preact"] else (y,)
    dz = st["dy"].double()
    if case["act"] != "none":
        z = st["preact"].double().requires_grad_(True)
        dz, = torch.autograd.grad(fn(z), z, dz)
    dx, dW = torch.einsum("mn,nk->mk", dz, W), torch.einsum("mn,mk->nk", dz, x)
    return (dx, dW, dz.sum(0)) if case["bias"] else (dx, dW)
