"""The feed-forward block's operators, as measured cases: the gated projections and
their backward pass, and the norms around a block fused with its gate, its scales
and the residual stream, with their backward pass.

``own`` False: elementary torch operations in 32 bits, rounded once at the end.
``own`` True: the calls a user makes of dense_gemm_blackwell_sm_gb300.ffn.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # one decoded token through the largest projection shape (14336 x 4096): the weight stream is all there is
        {"name": "gated token 1x14336x4096 bf16", "op": "gated", "M": 1, "F": 14336, "K": 4096, "dtype": "bf16",
         "act": "silu", "save": False},
        # a decode batch of eight on the square projection: the smallest call, launch and latency count
        {"name": "gated batch 8x4096x4096 f16", "op": "gated", "M": 8, "F": 4096, "K": 4096, "dtype": "f16",
         "act": "gelu_tanh", "save": False},
        # a short ragged training batch of a small model, pre-activations kept for the backward pass
        {"name": "gated ragged 300x1541x520 bf16", "op": "gated", "M": 300, "F": 1541, "K": 520, "dtype": "bf16",
         "act": "gelu_erf", "save": True},
        # a full prompt of 8192 tokens through the projection shape: compute bound
        {"name": "gated prompt 8192x14336x4096 bf16", "op": "gated", "M": 8192, "F": 14336, "K": 4096,
         "dtype": "bf16", "act": "silu", "save": False},
        # backward of a small odd-sized layer from kept pre-activations, half precision
        {"name": "gated grad 777x1097x1032 f16", "op": "gated_grad", "M": 777, "F": 1097, "K": 1032, "dtype": "f16",
         "act": "gelu_tanh", "saved": True},
        # backward of a mid-sized layer that keeps nothing: the pre-activations are computed again
        {"name": "gated grad again 1024x4096x4096", "op": "gated_grad", "M": 1024, "F": 4096, "K": 4096,
         "dtype": "bf16", "act": "silu", "saved": False},
        # backward of a training batch through the projection shape: compute bound
        {"name": "gated grad 4096x14336x4096 bf16", "op": "gated_grad", "M": 4096, "F": 14336, "K": 4096,
         "dtype": "bf16", "act": "silu", "saved": True},
        # one decoded token: residual add and the next block's norm, pure latency
        {"name": "norm token 1x4096 bf16", "op": "norm", "M": 1, "D": 4096, "dtype": "bf16", "param": "bf16",
         "kind": "rms", "post": False, "groups": 0, "affine": True},
        # a prompt: norm after the block, per-channel layer scale, residual, norm before the next block
        {"name": "norm prompt 8192x4096 bf16", "op": "norm", "M": 8192, "D": 4096, "dtype": "bf16", "param": "f32",
         "kind": "rms", "post": True, "groups": 1, "affine": True},
        # a conditioned model (a gate for each sequence of 125 rows), odd width, single precision
        {"name": "norm gates 1000x1001 f32", "op": "norm", "M": 1000, "D": 1001, "dtype": "f32", "param": "f32",
         "kind": "layer", "post": True, "groups": 8, "affine": True},
        # the training batch's backward through both norms, the layer scale and the residual
        {"name": "norm grad 8192x4096 bf16", "op": "norm_grad", "M": 8192, "D": 4096, "dtype": "bf16",
         "param": "f32", "kind": "rms", "post": True, "groups": 1, "affine": True},
        # backward of the conditioned model, a gate for each sequence of 103 rows, odd width, half precision
        {"name": "norm grad gates 515x1023 f16", "op": "norm_grad", "M": 515, "D": 1023, "dtype": "f16",
         "param": "f16", "kind": "layer", "post": True, "groups": 5, "affine": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated", "gated_grad", "norm", "norm_grad"])
    if op == "gated":
        return {"op": op, "M": _log(rng, 1, 8192), "F": _log(rng, 256, 14336), "K": 8 * _log(rng, 32, 512),
                "dtype": rng.choice(["bf16", "f16"]), "act": rng.choice(["silu", "gelu_tanh", "gelu_erf", "relu"]),
                "save": rng.random() < 0.4}
    if op == "gated_grad":
        saved = rng.random() < 0.6
        return {"op": op, "M": _log(rng, 64, 4096 if saved else 2700), "F": _log(rng, 256, 14336),
                "K": 8 * _log(rng, 32, 512), "dtype": rng.choice(["bf16", "f16"]),
                "act": rng.choice(["silu", "gelu_tanh", "gelu_erf", "relu"]), "saved": saved}
    groups = rng.choice([0, 1, 1, 3, 16])
    per = max(1, _log(rng, 1, 8192) // max(1, groups))
    M = per * max(1, groups)
    if op == "norm_grad":
        M = max(1, groups) * max(per, 2)
    return {"op": op, "M": M, "D": _log(rng, 64, 8192) if M <= 4096 else _log(rng, 64, 4096),
            "dtype": rng.choice(["bf16", "f16", "f32"]), "param": "f32", "kind": rng.choice(["rms", "layer"]),
            "post": rng.random() < 0.6, "groups": groups, "affine": rng.random() < 0.8}


def work(case):
    if case["op"] in ("gated", "gated_grad"):
        M, F, K = case["M"], case["F"], case["K"]
        if case["op"] == "gated":
            return {"bytes": 2 * (M * K + 2 * F * K + M * F * (3 if case["save"] else 1)), "flops": 4 * M * F * K}
        # x, w and dh read, dx and dw written; the kept pre-activations read, or both products made again
        n = 2 * M * K + 4 * F * K + M * F + (2 * M * F if case["saved"] else 0)
        return {"bytes": 2 * n, "flops": (8 if case["saved"] else 12) * M * F * K}
    M, D, e = case["M"], case["D"], 4 if case["dtype"] == "f32" else 2
    p = 4 if case["param"] == "f32" else 2
    vectors = (2 if case["kind"] == "layer" else 1) * (2 if case["post"] else 1) if case["affine"] else 0
    if case["op"] == "norm":
        return {"bytes": 4 * M * D * e + (vectors + case["groups"]) * D * p, "flops": 12 * M * D}
    weights = vectors // 2 if case["kind"] == "layer" else vectors  # biases are not read, only their gradients written
    y = 1 if case["post"] or case["groups"] else 0
    return {"bytes": (5 + y) * M * D * e + (weights + case["groups"]) * D * p + (vectors + case["groups"]) * D * 4,
            "flops": 24 * M * D}


def _make(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DT[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, to=dt):
        v = torch.randn(shape, generator=g, device="cuda")
        return v.mul_(std).add_(mean).to(to)

    if case["op"] in ("gated", "gated_grad"):
        M, F, K = case["M"], case["F"], case["K"]
        s = {"x": normal(M, K), "w": normal(2 * F, K, std=0.02 * math.sqrt(4096 / K))}  # pre-activations of order one
        if case["op"] == "gated_grad":
            s["dh"] = normal(M, F, std=0.5)
            s["gu"] = normal(M, 2 * F, std=1.28) if case["saved"] else None
        return s
    M, D, pt = case["M"], case["D"], DT[case["param"]]
    vec = (lambda mean: normal(D, std=0.2, mean=mean, to=pt)) if case["affine"] else (lambda mean: None)
    layer = case["kind"] == "layer"
    s = {"y": normal(M, D, std=1.5, mean=0.25), "pre_weight": vec(1.0), "pre_bias": vec(0.0) if layer else None,
         "post_weight": vec(1.0) if case["post"] else None,
         "post_bias": vec(0.0) if case["post"] and layer else None,
         "gate": normal(case["groups"], D, std=0.3, mean=0.5, to=pt) if case["groups"] else None}
    if case["op"] == "norm":
        s["residual"] = normal(M, D, std=3.0)
        s["residual"][:, :: max(1, D // 7)] *= 8  # a stream's few large channels
    else:
        s["stream"] = normal(M, D, std=3.0, mean=0.1)
        s["ds"] = normal(M, D, std=0.5)
        s["dn"] = normal(M, D, std=0.5)
    return s


def prepare(case, seed):
    return dict(_make(case, seed), case=case)


# ---------------------------------------------------------------- plain forms


def _act(name, g):
    """The activation and its derivative."""
    if name == "relu":
        p = (g > 0).float()
        return g * p, p
    if name == "silu":
        p = 1 / (1 + torch.exp(-g))
        return g * p, p * (1 + g * (1 - p))
    if name == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (g + 0.044715 * g * g * g))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)
    p = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
    return g * p, p + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))


def _plain_gated(s, c):
    dt = s["x"].dtype
    gu = s["x"].float() @ s["w"].float().t()
    h = _act(c["act"], gu[:, : c["F"]])[0] * gu[:, c["F"]:]
    return (h.to(dt), gu.to(dt)) if c["save"] else h.to(dt)


def _plain_gated_grad(s, c):
    dt = s["x"].dtype
    x, w, dh = s["x"].float(), s["w"].float(), s["dh"].float()
    gu = s["gu"].float() if c["saved"] else x @ w.t()
    a, slope = _act(c["act"], gu[:, : c["F"]])
    dgu = torch.cat([dh * gu[:, c["F"]:] * slope, dh * a], 1)
    return (dgu @ w).to(dt), (dgu.t() @ x).to(dt)


def _unit(v, kind):
    """The row's normalised values and its reciprocal deviation."""
    v = v - v.mean(1, keepdim=True) if kind == "layer" else v
    r = torch.rsqrt(v.square().mean(1, keepdim=True) + EPS)
    return v * r, r


def _affine(v, weight, bias):
    v = v if weight is None else v * weight.float()
    return v if bias is None else v + bias.float()


def _rows(gate, M):
    return gate.float().repeat_interleave(M // gate.shape[0], 0)


def _plain_norm(s, c):
    dt = s["y"].dtype
    z = s["y"].float()
    if c["post"]:
        z = _affine(_unit(z, c["kind"])[0], s["post_weight"], s["post_bias"])
    if c["groups"]:
        z = z * _rows(s["gate"], c["M"])
    t = s["residual"].float() + z
    n = _affine(_unit(t, c["kind"])[0], s["pre_weight"], s["pre_bias"])
    return t.to(dt), n.to(dt)


def _unit_grad(d, v, weight, kind):
    """Gradients of the norm's input, weight and bias."""
    u, r = _unit(v, kind)
    a = d if weight is None else d * weight.float()
    dv = a - u * (a * u).mean(1, keepdim=True)
    if kind == "layer":
        dv = dv - a.mean(1, keepdim=True)
    return dv * r, (d * u).sum(0), d.sum(0)


def _plain_norm_grad(s, c):
    dt = s["y"].dtype
    layer = c["kind"] == "layer"
    y = s["y"].float()
    t, pre_w, pre_b = _unit_grad(s["dn"].float(), s["stream"].float(), s["pre_weight"], c["kind"])
    t = t + s["ds"].float()
    z = _affine(_unit(y, c["kind"])[0], s["post_weight"], s["post_bias"]) if c["post"] else y
    dz, dgate = t, None
    if c["groups"]:
        dz = t * _rows(s["gate"], c["M"])
        dgate = (t * z).view(c["groups"], -1, c["D"]).sum(1)
    dy, post_w, post_b = _unit_grad(dz, y, s["post_weight"], c["kind"]) if c["post"] else (dz, None, None)
    affine = c["affine"]
    return (t.to(dt), dy.to(dt), dgate, post_w if affine else None, post_b if affine and layer else None,
            pre_w if affine else None, pre_b if affine and layer else None)


def run(state):
    c = state["case"]
    if not own:
        return {"gated": _plain_gated, "gated_grad": _plain_gated_grad, "norm": _plain_norm,
                "norm_grad": _plain_norm_grad}[c["op"]](state, c)
    from dense_gemm_blackwell_sm_gb300 import ffn

    if c["op"] == "gated":
        return ffn.gated(state["x"], state["w"], act=c["act"], save=c["save"])
    if c["op"] == "gated_grad":
        return ffn.gated_backward(state["dh"], state["x"], state["w"], gu=state["gu"], act=c["act"])
    shared = dict(post_norm=c["post"], post_weight=state["post_weight"], gate=state["gate"],
                  pre_weight=state["pre_weight"], kind=c["kind"], eps=EPS)
    if c["op"] == "norm":
        return ffn.block_norm(state["y"], state["residual"], post_bias=state["post_bias"],
                              pre_bias=state["pre_bias"], **shared)
    return tuple(ffn.block_norm_backward(state["ds"], state["dn"], state["y"], state["stream"],
                                         post_bias=state["post_bias"], pre_bias=state["pre_bias"], **shared))


# ------------------------------------------------- the definitions in 64 bits


def _exact_act(name, g):
    if name == "relu":
        return torch.clamp(g, min=0)
    if name == "silu":
        return g * torch.sigmoid(g)
    if name == "gelu_tanh":
        # (1 + tanh(v)) / 2 is the logistic function of 2 v
        return g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))
    return g * 0.5 * torch.erfc(-g / math.sqrt(2))


def _exact_norm(v, weight, bias, kind):
    if kind == "layer":
        var, mean = torch.var_mean(v, dim=1, unbiased=False, keepdim=True)
        v = (v - mean) / torch.sqrt(var + EPS)
    else:
        v = v / torch.sqrt((v * v).sum(1, keepdim=True) / v.shape[1] + EPS)
    if weight is not None:
        v = v * weight
    return v if bias is None else v + bias


def exact(case, seed):
    c = case
    s = {k: v.double() if v is not None else None for k, v in _make(case, seed).items()}
    if c["op"] == "gated":
        gate, up = s["w"].split(c["F"])
        g, u = s["x"] @ gate.t(), s["x"] @ up.t()
        h = _exact_act(c["act"], g) * u
        return (h, torch.cat([g, u], 1)) if c["save"] else h
    if c["op"] == "gated_grad":
        gu = s["gu"] if c["saved"] else s["x"] @ s["w"].t()
        gu = gu.requires_grad_()
        g, u = gu.split(c["F"], 1)
        dgu, = torch.autograd.grad(_exact_act(c["act"], g) * u, gu, s["dh"])
        return dgu @ s["w"], dgu.t() @ s["x"]

    def merged(y, gate, post_weight, post_bias):
        z = _exact_norm(y, post_weight, post_bias, c["kind"]) if c["post"] else y
        if gate is None:
            return z
        return (z.view(c["groups"], -1, c["D"]) * gate[:, None]).view(c["M"], c["D"])

    if c["op"] == "norm":
        t = s["residual"] + merged(s["y"], s["gate"], s["post_weight"], s["post_bias"])
        return t, _exact_norm(t, s["pre_weight"], s["pre_bias"], c["kind"])
    leaf = {k: v.requires_grad_() for k, v in s.items() if v is not None and k not in ("ds", "dn")}
    n = _exact_norm(leaf["stream"], leaf.get("pre_weight"), leaf.get("pre_bias"), c["kind"])
    pre = [k for k in ("stream", "pre_weight", "pre_bias") if k in leaf]
    got = dict(zip(pre, torch.autograd.grad(n, [leaf[k] for k in pre], s["dn"])))
    total = got["stream"] + s["ds"]
    z = merged(leaf["y"], leaf.get("gate"), leaf.get("post_weight"), leaf.get("post_bias"))
    post = [k for k in ("y", "gate", "post_weight", "post_bias") if k in leaf]
    got.update(zip(post, torch.autograd.grad(z, [leaf[k] for k in post], total) if z.requires_grad else ()))
    return (total, got["y"], got.get("gate"), got.get("post_weight"), got.get("post_bias"),
            got.get("pre_weight"), got.get("pre_bias"))
