"""What is measured of the operators around the expert path: scored routing, layer
norm and the linear product with a fused epilogue, each forward and backward.

`run` computes them in plain torch operations, or, with `own` set, through the
framework's entry points; `exact` gives the definition's values in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SCORES = ("softmax", "sigmoid")  # in the order of the library's score codes
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")  # in the order of its activation codes
EPS = 1e-5


def listed():
    return [
        # a decoding step's routing at the Qwen3-30B-A3B layer: 8 tokens, softmax over all 128 experts
        dict(name="route decode t8", op="route_fwd", T=8, E=128, k=8, score="softmax", bias=False, groups=1, top_groups=1,
             group_top=1, renorm=True, scale=1.0),
        # a training batch on a layer balanced by a selection bias, experts in 8 groups of which 4 are used
        dict(name="route groups t16384", op="route_fwd", T=16384, E=256, k=8, score="sigmoid", bias=True, groups=8,
             top_groups=4, group_top=2, renorm=True, scale=2.5),
        # the same batch on a softmax layer that does not renormalise: the gradient reaches every logit
        dict(name="route bwd softmax t16384", op="route_bwd", T=16384, E=128, k=8, score="softmax", renorm=False, scale=1.0),
        # a ragged batch on the sigmoid layer
        dict(name="route bwd sigmoid t2047", op="route_bwd", T=2047, E=256, k=8, score="sigmoid", renorm=True, scale=2.5),
        # the norm in front of the router: decoding, and a large batch at the GLM-4.5-Air width
        dict(name="norm decode t8", op="norm_fwd", T=8, H=2048, dtype="bf16"),
        dict(name="norm t16384", op="norm_fwd", T=16384, H=4096, dtype="bf16"),
        # its backward in training, and an fp32 layer of an odd batch and a width that is no multiple of a wave's stride
        dict(name="norm bwd t8192", op="norm_bwd", T=8192, H=4096, dtype="bf16"),
        dict(name="norm bwd f32 t1023", op="norm_bwd", T=1023, H=2880, dtype="f32"),
        # a shared expert's down product, decoding: the routed sum is its residual
        dict(name="linear decode t8", op="linear_fwd", T=8, I=768, O=2048, dtype="bf16", act="none", bias=True, mul=False,
             residual=True, save=False),
        # a shared expert's first product over a ragged training batch: bias and activation, z kept for the backward
        dict(name="linear t4099", op="linear_fwd", T=4099, I=2048, O=768, dtype="bf16", act="gelu", bias=True, mul=False,
             residual=False, save=True),
        # the backward of a gated shared expert's gate product at the GLM-4.5-Air shape
        dict(name="linear bwd t8192", op="linear_bwd", T=8192, I=4096, O=1408, dtype="bf16", act="silu", bias=False, mul=True),
        # an fp32 layer of odd sizes
        dict(name="linear bwd f32 t333", op="linear_bwd", T=333, I=200, O=136, dtype="f32", act="gelu_tanh", bias=True,
             mul=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    return 8 * _log_int(rng, lo // 8, hi // 8)


def draw(rng):
    op = rng.choice(("route_fwd", "route_bwd", "norm_fwd", "norm_bwd", "linear_fwd", "linear_bwd"))
    if op.startswith("route"):
        E = rng.choice((rng.randint(2, 256), 16 * rng.randint(1, 16), 128, 256))
        c = dict(op=op, T=_log_int(rng, 1, 16384), E=E, k=rng.randint(1, min(16, E)), score=rng.choice(SCORES),
                 renorm=rng.random() < 0.6, scale=rng.choice((1.0, 2.5)))
        if op == "route_bwd":
            # one renormalised weight is constant: its gradient is zero, and nothing to compare
            return dict(c, k=max(c["k"], 2)) if c["renorm"] else c
        groups = rng.choice([g for g in range(1, 17) if E % g == 0])
        size = E // groups
        top = rng.randint(-(-c["k"] // size), groups)
        return dict(c, bias=rng.random() < 0.6, groups=groups, top_groups=top, group_top=rng.choice((1, 2)) if size > 1 else 1)
    dtype = "bf16" if rng.random() < 0.7 else "f32"
    if op.startswith("norm"):
        T, H = _log_int(rng, 1, 16384), _width(rng, 64, 8192)
        return dict(op=op, T=max(1, min(T, (1 << 26) // H)), H=H, dtype=dtype)
    T, I, O = _log_int(rng, 1, 8192), _width(rng, 64, 4096), _width(rng, 64, 4096)
    if dtype == "f32":
        T = max(1, min(T, (1 << 31) // (I * O)))  # fp32 products are the small layers'
    T = max(1, min(T, (1 << 35) // (I * O)))
    c = dict(op=op, T=T, I=I, O=O, dtype=dtype, act=rng.choice(ACTS), bias=rng.random() < 0.5, mul=rng.random() < 0.3)
    return c if op == "linear_bwd" else dict(c, residual=rng.random() < 0.5, save=rng.random() < 0.5)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op, T = case["op"], case["T"]
    s = {"case": case}

    def normal(name, *shape, dtype=torch.float32, scale=1.0, shift=0.0):
        s[name] = (torch.randn(*shape, generator=g, device=dev) * scale + shift).to(dtype)

    def room(name, *shape, dtype):
        s[name] = torch.empty(*shape, dtype=dtype, device=dev)

    if op.startswith("route"):
        E, k = case["E"], case["k"]
        # the spread of a trained router's logits, some experts hotter than others
        normal("logits", T, E)
        s["logits"] += 0.5 * torch.randn(E, generator=g, device=dev)
        room("idx", T, k, dtype=torch.int32)
        if op == "route_fwd":
            normal("bias", E, scale=0.05)
            if not case["bias"]:
                s["bias"] = None
            room("w", T, k, dtype=torch.float32)
        else:
            s["idx"].copy_(torch.rand(T, E, generator=g, device=dev).argsort(1)[:, :k])
            normal("dg", T, k)
            room("dlogits", T, E, dtype=torch.float32)
        return s
    d = DTYPES[case["dtype"]]
    if op.startswith("norm"):
        H = case["H"]
        normal("x", T, H, dtype=d, scale=2.0, shift=0.25)
        normal("gamma", H, dtype=d, scale=0.2, shift=1.0)
        normal("beta", H, dtype=d, scale=0.2)
        room("mean", T, dtype=torch.float32)
        room("rstd", T, dtype=torch.float32)
        if op == "norm_fwd":
            room("y", T, H, dtype=d)
        else:
            x64 = s["x"].double()
            s["mean"].copy_(x64.mean(1))
            s["rstd"].copy_((x64.var(1, unbiased=False) + EPS).rsqrt())
            normal("dy", T, H, dtype=d)
            room("dx", T, H, dtype=d)
            room("dgamma", H, dtype=d)
            room("dbeta", H, dtype=d)
        return s
    I, O = case["I"], case["O"]
    normal("x", T, I, dtype=d)
    normal("w", I, O, dtype=d, scale=I ** -0.5)
    if case["mul"]:
        normal("mul", T, O, dtype=d)
    if op == "linear_fwd":
        if case["bias"]:
            normal("b", O, dtype=d, scale=0.2)
        if case["residual"]:
            normal("residual", T, O, dtype=d)
        if case["save"]:
            room("z", T, O, dtype=d)
        room("y", T, O, dtype=d)
    else:
        if case["act"] != "none" or case["mul"]:
            normal("z", T, O, dtype=d)
            room("dz", T, O, dtype=d)
        normal("dy", T, O, dtype=d)
        room("dx", T, I, dtype=d)
        room("dw", I, O, dtype=d)
        if case["bias"]:
            room("db", O, dtype=d)
        if case["mul"]:
            room("dmul", T, O, dtype=d)
    return s


def run(s):
    return _own(s) if own else _PLAIN[s["case"]["op"]](s)


def _own(s):
    """The calls of a program that keeps its buffers: outputs in the state, the workspace made once."""
    from expert_grouped_gemm_top_amd import moe

    c, get = s["case"], s.get
    op = c["op"]
    if op == "route_fwd":
        moe.moe_route_scored(s["logits"], s["bias"], s["idx"], s["w"], c["k"], score=SCORES.index(c["score"]),
                             n_groups=c["groups"], top_groups=c["top_groups"], group_top=c["group_top"],
                             renormalize=c["renorm"], scale=c["scale"])
        return s["idx"], s["w"]
    if op == "route_bwd":
        moe.moe_route_scored_bwd(s["logits"], s["idx"], s["dg"], s["dlogits"], score=SCORES.index(c["score"]),
                                 renormalize=c["renorm"], scale=c["scale"])
        return s["dlogits"]
    if op == "norm_fwd":
        moe.moe_layernorm_fwd(s["x"], s["gamma"], s["beta"], s["y"], s["mean"], s["rstd"], eps=EPS)
        return s["y"], s["mean"], s["rstd"]
    if "ws" not in s:
        need = (moe.moe_layernorm_workspace_bytes(c["T"], c["H"]) if op == "norm_bwd" else
                moe.moe_linear_workspace_bytes(c["T"], c["I"], c["O"], s["x"].dtype))
        s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device=s["x"].device)
    if op == "norm_bwd":
        moe.moe_layernorm_bwd(s["x"], s["gamma"], s["mean"], s["rstd"], s["dy"], s["dx"], s["dgamma"], s["dbeta"], s["ws"])
        return s["dx"], s["dgamma"], s["dbeta"]
    act = ACTS.index(c["act"])
    if op == "linear_fwd":
        moe.moe_linear_fwd(s["x"], s["w"], get("b"), s["y"], act=act, mul=get("mul"), residual=get("residual"),
                           z_save=get("z"), workspace=s["ws"])
        return (s["y"], s["z"]) if c["save"] else s["y"]
    moe.moe_linear_bwd(s["x"], s["w"], s["dy"], get("dz"), s["dx"], s["dw"], dbias=get("db"), act=act, z=get("z"),
                       mul=get("mul"), dmul=get("dmul"), workspace=s["ws"])
    return [s[n] for n in ("dx", "dw", "db", "dmul") if n in s]


# ---- the plain forms ----------------------------------------------------------


def _scores(l, kind):
    if kind == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    e = torch.exp(l - l.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _route_fwd(s):
    """In 64 bits: choices next to a border are decided by more than fp32 holds."""
    c = s["case"]
    T, E, G, k = c["T"], c["E"], c["groups"], c["k"]
    l = s["logits"].double()
    p = _scores(l, c["score"])
    choice = p if s["bias"] is None else p + s["bias"].double()
    if G > 1:
        best = choice.view(T, G, E // G).sort(dim=2, descending=True)[0][:, :, :c["group_top"]].sum(2)
        keep = best.sort(dim=1, descending=True, stable=True)[1][:, :c["top_groups"]]
        kept = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, keep, True)
        choice = torch.where(kept.repeat_interleave(E // G, 1), choice, -math.inf)
    idx = choice.sort(dim=1, descending=True, stable=True)[1][:, :k]
    w = p.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return idx.int(), (c["scale"] * w).float()


def _route_bwd(s):
    c = s["case"]
    idx = s["idx"].long()
    p = _scores(s["logits"], c["score"])
    sel, g = p.gather(1, idx), c["scale"] * s["dg"]
    if c["renorm"]:
        total = sel.sum(1, keepdim=True)
        g = (g - (g * sel).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(p).scatter_(1, idx, g)
    if c["score"] == "sigmoid":
        return ds * p * (1.0 - p)
    return p * (ds - (ds * p).sum(1, keepdim=True))


def _norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    x = x - mean
    rstd = 1.0 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
    y = x * rstd * s["gamma"].float() + s["beta"].float()
    return y.to(s["x"].dtype), mean.view(-1), rstd.view(-1)


def _norm_bwd(s):
    d = s["x"].dtype
    dy, r = s["dy"].float(), s["rstd"].view(-1, 1)
    xh = (s["x"].float() - s["mean"].view(-1, 1)) * r
    g = dy * s["gamma"].float()
    dx = r * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return dx.to(d), (dy * xh).sum(0).to(d), dy.sum(0).to(d)


def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))


def _act_slope(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        sg = 1.0 / (1.0 + torch.exp(-z))
        return sg * (1.0 + z * (1.0 - sg))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    a = math.sqrt(2.0 / math.pi)
    t = torch.tanh(a * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * a * (1.0 + 3 * 0.044715 * z * z)


def _linear_fwd(s):
    c, d = s["case"], s["x"].dtype
    z = s["x"].float() @ s["w"].float()
    if c["bias"]:
        z = z + s["b"].float()
    y = _act(z, c["act"])
    if c["mul"]:
        y = y * s["mul"].float()
    if c["residual"]:
        y = y + s["residual"].float()
    return (y.to(d), z.to(d)) if c["save"] else y.to(d)


def _linear_bwd(s):
    c, d = s["case"], s["x"].dtype
    dy = s["dy"].float()
    dz, dmul = dy, None
    if c["mul"]:
        dz, dmul = dy * s["mul"].float(), dy * _act(s["z"].float(), c["act"])
    if c["act"] != "none":
        dz = dz * _act_slope(s["z"].float(), c["act"])
    out = [dz @ s["w"].float().t(), s["x"].float().t() @ dz]
    if c["bias"]:
        out.append(dz.sum(0))
    if c["mul"]:
        out.append(dmul)
    return [o.to(d) for o in out]


_PLAIN = {"route_fwd": _route_fwd, "route_bwd": _route_bwd, "norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd,
          "linear_fwd": _linear_fwd, "linear_bwd": _linear_bwd}


# ---- what a pass cannot do without --------------------------------------------


def work(c):
    op, T = c["op"], c["T"]
    if op == "route_fwd":
        E = c["E"]
        return {"bytes": 4 * T * E + (4 * E if c["bias"] else 0) + 8 * T * c["k"], "flops": 8 * T * E}
    if op == "route_bwd":
        E, k = c["E"], c["k"]
        # all logits where the score's sum reaches every expert, else the selected ones
        reads = T * E if c["score"] == "softmax" and not c["renorm"] else T * k
        return {"bytes": 4 * (reads + T * E) + 8 * T * k, "flops": 8 * T * E}
    b = 2 if c["dtype"] == "bf16" else 4
    if op == "norm_fwd":
        return {"bytes": b * (2 * T + 2) * c["H"] + 8 * T, "flops": 8 * T * c["H"]}
    if op == "norm_bwd":
        return {"bytes": b * (3 * T + 3) * c["H"] + 8 * T, "flops": 14 * T * c["H"]}
    I, O = c["I"], c["O"]
    n = T * I + I * O + T * O + (O if c["bias"] else 0)  # x, w, y or dy, bias or its gradient
    if op == "linear_fwd":
        n += T * O * (c["mul"] + c["residual"] + c["save"])
        return {"bytes": b * n, "flops": 2 * T * I * O}
    n += T * I + I * O + (T * O if c["act"] != "none" or c["mul"] else 0) + 2 * T * O * c["mul"]  # dx, dw, z, mul and dmul
    return {"bytes": b * n, "flops": 4 * T * I * O}


# ---- the definitions in 64 bits -----------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("route"):
        out = (_exact_route if op == "route_fwd" else _exact_route_bwd)(case, s)
        return tuple(torch.from_numpy(o) for o in out) if isinstance(out, tuple) else torch.from_numpy(out)
    v = {n: t.double() for n, t in s.items() if isinstance(t, torch.Tensor)}
    if op == "norm_fwd":
        var, mean = torch.var_mean(v["x"], 1, unbiased=False)
        rstd = (var + EPS) ** -0.5
        return torch.addcmul(v["beta"], (v["x"] - mean[:, None]) * rstd[:, None], v["gamma"]), mean, rstd
    if op == "norm_bwd":
        H = case["H"]
        xh = (v["x"] - v["mean"][:, None]) * v["rstd"][:, None]
        g = v["dy"] * v["gamma"]
        along = torch.stack([g.sum(1), (g * xh).sum(1)], 1) / H  # the parts of g along 1 and along xh
        dx = v["rstd"][:, None] * (g - along[:, :1] - along[:, 1:] * xh)
        return dx, torch.linalg.vecdot(v["dy"], xh, dim=0), v["dy"].sum(0)
    value, slope = _ACT64[case["act"]]
    if op == "linear_fwd":
        z = torch.addmm(v["b"], v["x"], v["w"]) if case["bias"] else torch.mm(v["x"], v["w"])
        y = value(z)
        y = y * v["mul"] if case["mul"] else y
        y = y + v["residual"] if case["residual"] else y
        return (y, z) if case["save"] else y
    dz = v["dy"] * v["mul"] if case["mul"] else v["dy"]
    dz = dz * slope(v["z"]) if case["act"] != "none" else dz
    out = [torch.mm(dz, v["w"].t()), torch.mm(dz.t(), v["x"]).t()]
    out += [torch.mv(dz.t(), torch.ones(case["T"], dtype=dz.dtype, device=dz.device))] if case["bias"] else []
    return out + ([value(v["z"]) * v["dy"]] if case["mul"] else [])


def _phi(z):
    return 0.5 * torch.erfc(-z / math.sqrt(2.0))


def _u(z):
    return math.sqrt(8.0 / math.pi) * (z + 0.044715 * z ** 3)  # 0.5 (1 + tanh(u / 2)) = sigmoid(u)


_ACT64 = {
    "none": (lambda z: z, torch.ones_like),
    "relu": (lambda z: z.clamp(min=0), lambda z: torch.heaviside(z, torch.zeros_like(z))),
    "gelu": (lambda z: z * _phi(z), lambda z: _phi(z) + z * torch.exp(-z * z / 2) * (2 * math.pi) ** -0.5),
    "gelu_tanh": (lambda z: z * torch.sigmoid(_u(z)),
                  lambda z: torch.sigmoid(_u(z)) * (1 + z * torch.sigmoid(-_u(z)) * math.sqrt(8 / math.pi) * (1 + 0.134145 * z * z))),
    "silu": (lambda z: z * torch.sigmoid(z), lambda z: torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z)),
}


def _log_scores(l, kind):
    if kind == "sigmoid":
        return -np.logaddexp(0.0, -l)
    return l - np.logaddexp.reduce(l, axis=1, keepdims=True)


def _exact_route(c, s):
    l = s["logits"].double().cpu().numpy()
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    logs = _log_scores(l, c["score"])
    choice = np.exp(logs) + (0.0 if s["bias"] is None else s["bias"].double().cpu().numpy())
    size = E // G
    worth = -np.sort(-choice.reshape(T * G, size), axis=1)[:, :c["group_top"]].sum(1).reshape(T, G)
    rank = np.empty((T, G), np.int64)
    np.put_along_axis(rank, np.argsort(-worth, axis=1, kind="stable"), np.arange(G)[None], axis=1)
    choice[np.repeat(rank >= c["top_groups"], size, axis=1)] = -np.inf
    idx = np.argsort(-choice, axis=1, kind="stable")[:, :k]
    picked = np.take_along_axis(logs, idx, axis=1)
    if c["renorm"]:
        picked = picked - np.logaddexp.reduce(picked, axis=1, keepdims=True)
    return idx.astype(np.int32), c["scale"] * np.exp(picked)


def _exact_route_bwd(c, s):
    """d(log w_j)/dl written out: w_j times the difference of two of the log scores' slopes."""
    l, idx = s["logits"].double().cpu().numpy(), s["idx"].long().cpu().numpy()
    logs = _log_scores(l, c["score"])
    picked = np.take_along_axis(logs, idx, axis=1)
    if c["renorm"]:
        picked = picked - np.logaddexp.reduce(picked, axis=1, keepdims=True)
    v = c["scale"] * np.exp(picked) * s["dg"].double().cpu().numpy()  # w_j dg_j
    out = np.zeros_like(l)
    if c["renorm"]:
        v = v - np.exp(picked) * v.sum(1, keepdims=True)  # of the log scores of the selected
    np.put_along_axis(out, idx, v, axis=1)
    if c["score"] == "sigmoid":
        return out * np.exp(_log_scores(-l, "sigmoid"))
    return out - np.exp(logs) * v.sum(1, keepdims=True)
