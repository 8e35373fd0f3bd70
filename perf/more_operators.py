"""What is measured of the operators behind the block in a training step: the routers'
balance loss, softmax cross entropy over a vocabulary without kept logits, each
forward and backward, and AdamW over many tensors with states of 32 or 8 bits.

`run` computes them in plain torch operations, or, with `own` set, through the
framework's entry points; `exact` gives the definition's values in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SCORES = ("softmax", "sigmoid")  # in the order of the library's score codes
BETA1, BETA2, ADAM_EPS, LR, SEED = 0.9, 0.999, 1e-8, 1e-3, 12345
BLOCK = 256  # elements that share a scale where states have 8 bits


def listed():
    return [
        # the balance loss of a small fine-tuning batch at the Qwen3-30B-A3B layer: one sequence, softmax scores
        dict(name="balance t128", op="balance_fwd", T=128, E=128, k=8, score="softmax", seqs=1, fill=1.0),
        # a training batch of ragged sequences, each balanced by itself, with padding behind the last; sigmoid scores
        dict(name="balance seqs t16384", op="balance_fwd", T=16384, E=256, k=8, score="sigmoid", seqs=8, fill=0.95),
        # its gradient on a softmax layer, added to the gradient that came from the routing weights
        dict(name="balance bwd t16384", op="balance_bwd", T=16384, E=128, k=8, score="softmax", seqs=1, fill=1.0, add=True),
        # the gradient of a ragged batch on the sigmoid layer
        dict(name="balance bwd seqs t2047", op="balance_bwd", T=2047, E=256, k=8, score="sigmoid", seqs=5, fill=0.9, add=False),
        # scoring the small fine-tuning batch: the head's weights are read for 128 tokens
        dict(name="vocab t128", op="vocab_fwd", T=128, H=2048, V=131072, pad=0, ignored=0.0, dtype="bf16"),
        # a fine-tuning batch in which the prompts' tokens carry no loss, over a vocabulary of an odd size
        dict(name="vocab t4096", op="vocab_fwd", T=4096, H=2048, V=131069, pad=3, ignored=0.4, dtype="bf16"),
        # the small batch's gradient under a frozen head
        dict(name="vocab bwd frozen t128", op="vocab_bwd", T=128, H=2048, V=131072, pad=0, ignored=0.25, dtype="bf16", dw=False,
             weighted=False),
        # full training at the GLM-4.5-Air width: both gradients
        dict(name="vocab bwd t8192", op="vocab_bwd", T=8192, H=4096, V=65536, pad=0, ignored=0.0, dtype="bf16", dw=True,
             weighted=False),
        # an fp32 model of odd sizes, tokens weighted one by one
        dict(name="vocab bwd f32 t333", op="vocab_bwd", T=333, H=200, V=1003, pad=5, ignored=0.2, dtype="f32", dw=True,
             weighted=True),
        # an adapter's step: many small tensors of odd sizes
        dict(name="adamw adapters", op="adamw", n=64, lo=17, hi=65537, dtype="f32", bits=32, master=False),
        # 32 of the Qwen3-30B-A3B layer's 128 experts, as a device of four holds them: bf16 weights with fp32 masters
        dict(name="adamw experts", op="adamw", n=3, lo=50331648, hi=50331648, dtype="bf16", bits=32, master=True),
        # the same with nothing but 8-bit states beside the bf16 weights
        dict(name="adamw experts 8 bits", op="adamw", n=3, lo=50331648, hi=50331648, dtype="bf16", bits=8, master=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("balance_fwd", "balance_bwd", "vocab_fwd", "vocab_bwd", "adamw", "adamw"))
    dtype = "bf16" if rng.random() < 0.7 else "f32"
    if op.startswith("balance"):
        E, T = rng.choice((rng.randint(2, 256), 128, 256)), _log_int(rng, 1, 16384)
        seqs = rng.choice((1, 1, rng.randint(1, min(T, 64))))
        c = dict(op=op, T=T, E=E, k=rng.randint(1, max(1, min(16, E - 1))), score=rng.choice(SCORES), seqs=seqs,
                 fill=rng.choice((1.0, round(rng.uniform(0.5, 1.0), 2))))
        return c if op == "balance_fwd" else dict(c, add=rng.random() < 0.5)
    if op.startswith("vocab"):
        H, V = 8 * _log_int(rng, 8, 512), _log_int(rng, 17, 131072)
        T = min(_log_int(rng, 1, 8192), (1 << 41 if dtype == "bf16" else 1 << 36) // (H * V))
        c = dict(op=op, T=max(1, T), H=H, V=V, pad=-V % 8, ignored=rng.choice((0.0, round(rng.uniform(0.0, 0.9), 2))), dtype=dtype)
        return c if op == "vocab_fwd" else dict(c, dw=rng.random() < 0.7, weighted=rng.random() < 0.4)
    n = _log_int(rng, 1, 200)
    hi = _log_int(rng, 1, (1 << 26) // n)
    return dict(op=op, n=n, lo=_log_int(rng, 1, hi), hi=hi, dtype=dtype, bits=rng.choice((32, 8)),
                master=dtype == "bf16" and rng.random() < 0.5)


def _sizes(c):
    """Elements of each tensor, from lo to hi in even steps of their logarithm."""
    n, lo, hi = c["n"], c["lo"], c["hi"]
    return [int(round(lo * (hi / lo) ** (i / max(1, n - 1)))) for i in range(n)]


def _counted(c):
    """Tokens that carry a loss."""
    return c["T"] - int(c["T"] * c["ignored"])


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = {"case": case}

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * scale).to(dtype)

    def room(*shape, dtype=torch.float32):
        return torch.zeros(*shape, dtype=dtype, device=dev)

    if case["op"].startswith("balance"):
        T, E, k, S = case["T"], case["E"], case["k"], case["seqs"]
        # the spread of a trained router's logits, some experts hotter than others
        s["logits"] = normal(T, E) + 0.5 * normal(E)
        idx = s["logits"].topk(k, dim=1)[1].int()
        end = max(1, int(T * case["fill"]))
        cuts = np.sort(np.random.default_rng(seed).integers(0, end + 1, S - 1))
        s["offsets"] = torch.tensor([0, *cuts.tolist(), end], dtype=torch.int32, device=dev)
        if case["op"] == "balance_fwd":
            s.update(idx=idx, counts=room(S, E, dtype=torch.int32), mean_p=room(S, E), loss=room(1))
        else:
            seq = torch.bucketize(torch.arange(T, device=dev, dtype=torch.int32), s["offsets"], right=True) - 1
            counts = room(S + 1, E, dtype=torch.int32)  # what the forward left; rows behind the last sequence apart
            counts.view(-1).index_add_(0, (seq.long()[:, None] * E + idx).reshape(-1), torch.ones(T * k, dtype=torch.int32, device=dev))
            # the gradient that is there is of the size of a routing weight's share
            s.update(counts=counts[:S].contiguous(), dlogits=room(T, E), dloss=1.0 + 0.1 * normal(1).abs(),
                     add=normal(T, E, scale=0.1 / T) if case["add"] else None)
        return s
    if case["op"].startswith("vocab"):
        T, H, V, d = case["T"], case["H"], case["V"], DTYPES[case["dtype"]]
        # logits of a trained model: a spread of 2, the target's raised by 0 to 12
        w = normal(H, V + case["pad"], scale=2.0 * H ** -0.5)
        y = torch.randint(0, V, (T,), generator=g, device=dev)
        at = w[:, y].t()
        lift = 12.0 * torch.rand(T, 1, generator=g, device=dev)
        s["x"] = (normal(T, H) + lift * at / (at * at).sum(1, keepdim=True)).to(d)
        s["w"] = w.to(d)
        y[torch.randperm(T, generator=g, device=dev)[:T - _counted(case)]] = -100
        s["target"] = y.int()
        del w, at
        if case["op"] == "vocab_fwd":
            s.update(loss=room(T), lse=room(T), mean=room(2))
            return s
        loss, lse = _exact_vocab(s["x"].double(), s["w"][:, :V], s["target"])  # what the forward left
        n = (s["target"] >= 0).sum()
        s.update(loss=loss.float(), lse=lse.float(), mean=torch.stack([loss.sum() / n.clamp(min=1), (n > 0) / n.clamp(min=1).double()]).float())
        s.update(dx=room(T, H, dtype=d), dw=room(H, V + case["pad"], dtype=d) if case["dw"] else None)
        s["dloss"] = torch.rand(T, generator=g, device=dev) / T if case["weighted"] else None
        return s
    # the tensors lie one behind the other, each from a multiple of BLOCK on
    sizes = _sizes(case)
    blocks = [-(-n // BLOCK) for n in sizes]
    starts = np.concatenate([[0], np.cumsum(blocks)])[:-1] * BLOCK
    total, d = int(sum(blocks)) * BLOCK, DTYPES[case["dtype"]]
    inside = torch.ones(total, dtype=torch.bool, device=dev)
    for at, n, b in zip(starts, sizes, blocks):
        inside[at + n:at + b * BLOCK] = False
    each = torch.exp(1.5 * normal(total // BLOCK)).repeat_interleave(BLOCK)  # gradients differ in size from row to row
    p = 0.02 * normal(total) * inside
    s["grad"] = (1e-3 * each * normal(total) * inside).to(d)
    m = 3e-4 * each * normal(total) * inside
    v = 1e-6 * each * each * torch.exp(0.5 * normal(total)) * inside
    del each
    s["param"] = p.to(d)
    s["master"] = p.to(d).float() + 1e-5 * normal(total) * inside if case["master"] else None
    if case["bits"] == 32:
        s.update(m=m, v=v, m_scale=None, v_scale=None)
    else:
        s["m"], s["m_scale"] = _to_codes(_encode_m, m.double(), 448.0, 0.5)
        s["v"], s["v_scale"] = _to_codes(_encode_v, v.double(), 1.75, 0.5)
    # every third tensor is of those that are not decayed (norms, biases)
    s["decay"] = [0.0 if i % 3 == 2 else 0.1 for i in range(len(sizes))]
    s["decays"] = torch.tensor(s["decay"], device=dev).repeat_interleave(torch.tensor(blocks, device=dev))
    s["parts"] = [(int(a), int(n)) for a, n in zip(starts, sizes)]
    s["counter"] = torch.tensor([10, 0], dtype=torch.int32, device=dev)
    s["lr"] = torch.full((1,), LR, device=dev)
    s["grad_scale"] = torch.full((1,), 0.75, device=dev)  # the clipping's factor
    return s


def run(s):
    return _own(s) if own else _PLAIN[s["case"]["op"]](s)


def _own(s):
    """The calls of a program that keeps its buffers: outputs in the state, workspaces and plans made once."""
    from expert_grouped_gemm_top_amd import moe

    c, dev = s["case"], torch.device("cuda")
    op = c["op"]

    def space(need):
        if "ws" not in s:
            s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
        return s["ws"]

    if op == "balance_fwd":
        moe.moe_balance_loss_fwd(s["logits"], s["idx"], s["counts"], s["mean_p"], s["loss"],
                                 space(moe.moe_balance_loss_workspace_bytes(c["T"], c["E"], c["seqs"])), alpha=0.01,
                                 score=SCORES.index(c["score"]), seq_offsets=s["offsets"])
        return s["counts"], s["mean_p"], s["loss"]
    if op == "balance_bwd":
        moe.moe_balance_loss_bwd(s["logits"], s["counts"], s["dlogits"], c["k"], alpha=0.01, score=SCORES.index(c["score"]),
                                 seq_offsets=s["offsets"], dloss=s["dloss"], dl_add=s["add"])
        return s["dlogits"]
    if op.startswith("vocab"):
        ws = space(moe.moe_vocab_loss_workspace_bytes(c["T"], c["H"], c["V"] + c["pad"], s["x"].dtype))
        if op == "vocab_fwd":
            moe.moe_vocab_loss_fwd(s["x"], s["w"], s["target"], s["loss"], s["lse"], s["mean"], ws, vocab=c["V"])
            return s["loss"], s["lse"], s["mean"]
        moe.moe_vocab_loss_bwd(s["x"], s["w"], s["target"], s["loss"], s["lse"], s["mean"], s["dx"], s["dw"], ws,
                               dloss=s["dloss"], vocab=c["V"])
        return (s["dx"], s["dw"]) if c["dw"] else s["dx"]
    if "plan" not in s:
        def cut(name, at, n, unit=1):
            return None if s[name] is None else s[name][at // unit:at // unit + -(-n // unit)]
        s["plan"] = moe.AdamWPlan([moe.AdamWTensor(
            cut("param", at, n), cut("grad", at, n), cut("m", at, n), cut("v", at, n), cut("m_scale", at, n, BLOCK),
            cut("v_scale", at, n, BLOCK), cut("master", at, n), decay) for (at, n), decay in zip(s["parts"], s["decay"])])
    moe.moe_adamw_step(s["plan"], s["counter"], s["lr"], beta1=BETA1, beta2=BETA2, eps=ADAM_EPS, grad_scale=s["grad_scale"],
                       seed=SEED)
    if c["bits"] == 32:
        return _adamw_outputs(s)
    if "moments" not in s:
        s["moments"] = [torch.empty(s["m"].shape, device=dev) for _ in range(2)]
    moe.moe_adamw_moments(s["m"], s["v"], s["m_scale"], s["v_scale"], *s["moments"])
    return [s["param"]] + ([s["master"]] if c["master"] else []) + s["moments"]


def _adamw_outputs(s):
    out = [s["param"]] + ([s["master"]] if s["master"] is not None else [])
    if s["case"]["bits"] == 32:
        return out + [s["m"], s["v"]]
    return out + [_decode(_value_m, s["m"], s["m_scale"]), _decode(_value_v, s["v"], s["v_scale"])]


# ---- the plain forms ----------------------------------------------------------


def _shares(l, score):
    """Each expert's share of its token's scores, and what a share's slope is multiplied by."""
    if score == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-l))
        return p / p.sum(1, keepdim=True), 1.0 / (1.0 + torch.exp(l))
    e = torch.exp(l - l.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True), torch.ones_like(l)


def _seq_of(s):
    """The sequence of every row; the number of sequences for the rows outside them."""
    T, S, o = s["case"]["T"], s["case"]["seqs"], s["offsets"]
    t = torch.arange(T, device=o.device, dtype=torch.int32)
    return torch.where((t >= o[0]) & (t < o[S]), (t[:, None] >= o[None, 1:]).sum(1), S)


def _balance_fwd(s):
    c = s["case"]
    E, S, o = c["E"], c["seqs"], s["offsets"]
    seq = _seq_of(s)
    p, _ = _shares(s["logits"], c["score"])
    n = (o[1:] - o[:-1]).double()
    of = (seq == torch.arange(S, device=o.device)[:, None]).float()
    hits = torch.zeros_like(p).scatter_add_(1, s["idx"].long(), torch.ones_like(p[:, :c["k"]]))
    total = (of @ torch.cat([p, hits], 1)).double()  # whole numbers below 2^24 stay what they are
    counts = total[:, E:].int()
    mean_p = total[:, :E] / n.clamp(min=1)[:, None]
    loss = 0.01 * E / c["k"] * (counts * mean_p).sum() / n.sum().clamp(min=1)
    return counts, mean_p.float(), loss.float().view(1)


def _balance_bwd(s):
    c = s["case"]
    S, o = c["seqs"], s["offsets"]
    seq = _seq_of(s)
    p, rest = _shares(s["logits"], c["score"])
    n = (o[1:] - o[:-1]).float()
    each = 0.01 * c["E"] / c["k"] * s["dloss"] / (n * n.sum()).clamp(min=1)
    inside = seq < S
    seq = seq.clamp(max=S - 1)
    cnt = s["counts"].float()[seq]
    d = each[seq][:, None] * p * rest * (cnt - (p * cnt).sum(1, keepdim=True))
    d = torch.where(inside[:, None], d, 0.0)
    return s["add"] + d if c["add"] else d


def _vocab_logits(s):
    c = s["case"]
    return s["x"].float() @ s["w"].float()[:, :c["V"]]


def _vocab_fwd(s):
    l, y = _vocab_logits(s), s["target"]
    top = l.amax(1, keepdim=True)
    keep = y >= 0
    lse = torch.log(torch.exp(l - top).sum(1)) + top[:, 0]
    loss = torch.where(keep, lse - l.gather(1, y.long().clamp(min=0)[:, None])[:, 0], 0.0)
    n = keep.sum()
    mean = torch.stack([loss.double().sum() / n.clamp(min=1), (n > 0) / n.clamp(min=1).double()])
    return loss, torch.where(keep, lse, 0.0), mean.float()


def _vocab_bwd(s):
    c, y, d = s["case"], s["target"], s["x"].dtype
    keep = y >= 0
    dz = torch.exp(_vocab_logits(s) - s["lse"][:, None])
    dz -= (torch.arange(c["V"], device=y.device, dtype=torch.int32) == y[:, None]).float()
    each = s["dloss"] if c["weighted"] else s["mean"][1]
    dz *= torch.where(keep, each, 0.0)[:, None]
    dx = (dz @ s["w"].float()[:, :c["V"]].t()).to(d)
    if not c["dw"]:
        return dx
    return dx, torch.nn.functional.pad((s["x"].float().t() @ dz).to(d), (0, c["pad"]))


def _mix(x):
    """A hash of 32 bits, held in 64."""
    x = ((x ^ (x >> 16)) * 0x85ebca77) & 0xffffffff
    x = ((x ^ (x >> 15)) * 0xc2b2ae3d) & 0xffffffff
    return x ^ (x >> 16)


def _dither(s, step, total):
    """32 bits for each element, from its place, the step and the seed."""
    key = _mix((_mix(step.long()) + SEED) & 0xffffffff)
    return _mix(torch.arange(total, device=step.device) ^ key)


def _share(h):
    """16 bits as a share of 1. The third keeps it away from values with which means of codes and gradients, tenths and
    thousandths of short binary numbers, would add up to whole steps but for their rounding."""
    return (h.double() + 1.0 / 3.0) / 65536


def _floor_to(a, step, u):
    """a >= 0 as multiples of `step`, up for the share u of what is left over."""
    return torch.floor(a / step + u)


def _binade(a):
    """The power of two at or below a > 0, 0 for 0 (the exponent's bits of a value of 64 bits)."""
    return (a.view(torch.int64) & 0x7ff0000000000000).view(torch.float64)


def _exponent(b):
    return (b.view(torch.int64) >> 52) - 1023


def _pow2(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _encode_m(a, u):
    """E4M3: sign, 4 bits of exponent, 3 of mantissa; a is at most 448 in size."""
    mag = a.abs()
    step = _binade(mag).clamp(min=2.0 ** -6) / 8
    got = _floor_to(mag, step, u) * step
    b = _binade(got).clamp(min=2.0 ** -6)
    normal = got >= 2.0 ** -6
    code = torch.where(normal, (_exponent(b) + 7) * 8 + (got / b - 1) * 8, got * 512)
    return (code + 128 * (a < 0)).to(torch.uint8)


def _value_m(q):
    mag = q & 127
    e, f = mag >> 3, (mag & 7).double()
    a = torch.where(e > 0, (8 + f) * _pow2(e - 10), f * 2.0 ** -9)
    return torch.where(q > 127, -a, a)


def _encode_v(a, u):
    """5 bits of exponent, 3 of mantissa, no sign; a is at most 1.75, and what is not zero stays so."""
    step = _binade(a).clamp(min=2.0 ** -31) / 8
    got = _floor_to(a, step, u) * step
    b = _binade(got).clamp(min=2.0 ** -31)
    code = (_exponent(b) + 31) * 8 + (got / b - 1) * 8
    return torch.where(a > 0, code.clamp(min=1), 0.0).to(torch.uint8)


def _value_v(q):
    return torch.where(q > 0, (8 + (q & 7).double()) * _pow2((q >> 3) - 34), 0.0)


def _to_codes(encode, a, most, u):
    """Codes of a, and each block's scale: the smallest power of two that keeps its largest, as fp32, within `most`."""
    top = a.abs().view(-1, BLOCK).amax(1).float().double()
    scale = _binade(top / most)
    scale = torch.where(scale * most < top, 2 * scale, scale).clamp(2.0 ** -126, 2.0 ** 127)
    return encode(a / scale.repeat_interleave(BLOCK), u), scale.float()


def _decode(value, q, scale):
    return (value(q.int()) * scale.double().repeat_interleave(BLOCK)).float()


def _round_bf16(p, r):
    """fp32 to bf16, up for the share of what is left over that 16 of the hash's bits say."""
    low = (r * 0x9e3779b1 & 0xffffffff) >> 16
    return ((p.view(torch.int32) + low.int()) & -65536).view(torch.float32).bfloat16()


def _adamw(s):
    c = s["case"]
    s["counter"][:1] += 1
    t = s["counter"][:1].double()
    small = c["bits"] == 8
    wide = torch.float64 if small else torch.float32  # codes next to a border are decided by more than fp32 holds
    g = s["grad"].to(wide) * s["grad_scale"].to(wide)
    m = _value_m(s["m"].int()) * s["m_scale"].double().repeat_interleave(BLOCK) if small else s["m"]
    v = _value_v(s["v"].int()) * s["v_scale"].double().repeat_interleave(BLOCK) if small else s["v"]
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    del g
    p = (s["param"] if s["master"] is None else s["master"]).float()
    lr = s["lr"].double()
    keep = (1 - lr * s["decays"].double()).float().repeat_interleave(BLOCK)
    step1, root2 = (lr / (1 - BETA1 ** t)).float(), torch.sqrt(1 - BETA2 ** t).float()
    p = p * keep - step1 * m.float() / (torch.sqrt(v.float()) / root2 + ADAM_EPS)
    del keep
    total = p.numel()
    r = _dither(s, s["counter"][:1], total) if small or (c["dtype"] == "bf16" and not c["master"]) else None
    if c["master"]:
        s["master"].copy_(p)
        s["param"].copy_(p)
    else:
        s["param"].copy_(p if c["dtype"] == "f32" else _round_bf16(p, r))
    if small:
        s["m"], s["m_scale"] = _to_codes(_encode_m, m, 448.0, _share(r & 0xffff))
        s["v"], s["v_scale"] = _to_codes(_encode_v, v, 1.75, _share(r >> 16))
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    return _adamw_outputs(s)


_PLAIN = {"balance_fwd": _balance_fwd, "balance_bwd": _balance_bwd, "vocab_fwd": _vocab_fwd, "vocab_bwd": _vocab_bwd,
          "adamw": _adamw}


# ---- what a pass cannot do without --------------------------------------------


def work(c):
    op = c["op"]
    if op.startswith("balance"):
        T, E, S = c["T"], c["E"], c["seqs"]
        if op == "balance_fwd":
            return {"bytes": 4 * T * (E + c["k"]) + 8 * S * E, "flops": 6 * T * E}
        return {"bytes": 4 * T * E * (2 + c["add"]) + 4 * S * E, "flops": 10 * T * E}
    if op.startswith("vocab"):
        b, n, H, V = (2 if c["dtype"] == "bf16" else 4), _counted(c), c["H"], c["V"]
        if op == "vocab_fwd":
            return {"bytes": b * (n * H + H * V) + 12 * c["T"], "flops": 2 * n * H * V}
        grads = b * c["T"] * H + (b * H * (V + c["pad"]) if c["dw"] else 0)
        return {"bytes": b * (n * H + H * V) + grads + 16 * c["T"], "flops": (6 if c["dw"] else 4) * n * H * V}
    n, b = sum(_sizes(c)), (2 if c["dtype"] == "bf16" else 4)
    # gradient and weight read, weight written; or master read and written and weight written
    each = b + (8 + b if c["master"] else 2 * b) + (16 if c["bits"] == 32 else 4 + 16 / BLOCK)
    return {"bytes": int(n * each), "flops": 16 * n}


# ---- the definitions in 64 bits -----------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("balance"):
        out = (_exact_balance if op == "balance_fwd" else _exact_balance_bwd)(case, s)
        return tuple(torch.from_numpy(np.ascontiguousarray(o)) for o in out) if isinstance(out, tuple) else torch.from_numpy(out)
    if op.startswith("vocab"):
        x, w, y = s["x"].double(), s["w"][:, :case["V"]], s["target"]
        if op == "vocab_fwd":
            loss, lse = _exact_vocab(x, w, y)
            n = max(1, _counted(case))
            return loss, lse, torch.stack([loss.sum() / n, torch.full_like(loss[0], min(_counted(case), 1) / n)])
        dx, dw = _exact_vocab_bwd(x, w, y, s["dloss"])
        return (dx, torch.cat([dw, dw.new_zeros(case["H"], case["pad"])], 1)) if case["dw"] else dx
    return _exact_adamw(case, s)


def _log_shares(l, kind):
    a = l if kind == "softmax" else -np.logaddexp(0.0, -l)
    return a - np.logaddexp.reduce(a, axis=1, keepdims=True)


def _exact_balance(c, s):
    E, S = c["E"], c["seqs"]
    p = np.exp(_log_shares(s["logits"].double().cpu().numpy(), c["score"]))
    o, idx = s["offsets"].cpu().numpy(), s["idx"].cpu().numpy()
    counts, mean = np.zeros((S, E), np.int32), np.zeros((S, E))
    for i in range(S):
        if o[i + 1] > o[i]:
            counts[i] = np.bincount(idx[o[i]:o[i + 1]].ravel(), minlength=E)
            mean[i] = p[o[i]:o[i + 1]].mean(0)
    return counts, mean, np.array([0.01 * E / c["k"] / (o[S] - o[0]) * np.vdot(counts, mean)])


def _exact_balance_bwd(c, s):
    """By the slopes of the log shares: d(log p_e)/dl_j = ([e = j] - p_j) sigma'(l_j)/sigma(l_j)."""
    l, o, counts = s["logits"].double().cpu().numpy(), s["offsets"].cpu().numpy(), s["counts"].cpu().numpy()
    logs = _log_shares(l, c["score"])
    out = s["add"].double().cpu().numpy().copy() if c["add"] else np.zeros_like(l)
    slope = 1.0 if c["score"] == "softmax" else np.exp(-np.logaddexp(0.0, l))
    for i in range(c["seqs"]):
        at = slice(o[i], o[i + 1])
        if o[i + 1] == o[i]:
            continue
        n = int(o[i + 1] - o[i])
        p = np.exp(logs[at])
        pull = p * counts[i]  # d loss / d log p_e, but for its factor
        d = pull - p * pull.sum(1, keepdims=True)
        out[at] += float(s["dloss"]) * 0.01 * c["E"] / c["k"] / n / float(o[-1] - o[0]) * d * (slope if np.isscalar(slope) else slope[at])
    return out


def _exact_vocab(x, w, y):
    """Losses and log sums in 64 bits, a run of tokens at a time."""
    loss, lse = torch.zeros(len(y), dtype=torch.float64, device=x.device), torch.zeros(len(y), dtype=torch.float64, device=x.device)
    w = w.double()
    for a in range(0, len(y), 2048):
        l = torch.mm(x[a:a + 2048], w)
        t = y[a:a + 2048].long()
        z = torch.logsumexp(l, 1)
        lse[a:a + 2048] = z.masked_fill(t < 0, 0.0)
        loss[a:a + 2048] = (z - l.gather(1, t.clamp(min=0)[:, None])[:, 0]).masked_fill(t < 0, 0.0)
    return loss, lse


def _exact_vocab_bwd(x, w, y, dloss):
    w = w.double()
    rows = torch.nonzero(y >= 0)[:, 0]
    dx, dw = torch.zeros_like(x), torch.zeros(w.shape, dtype=torch.float64, device=x.device)
    for a in range(0, len(rows), 2048):
        at = rows[a:a + 2048]
        dz = torch.softmax(torch.mm(x[at], w), 1)
        dz[torch.arange(len(at), device=x.device), y[at].long()] -= 1.0
        dz *= (torch.full_like(at, 1.0, dtype=torch.float64) / len(rows) if dloss is None else dloss[at].double())[:, None]
        dx[at] = torch.mm(dz, w.t())
        dw.addmm_(x[at].t(), dz)
    return dx, dw


def _table(kind):
    """Every value that a code of 8 bits stands for, those without a sign."""
    c = np.arange(1, 127 if kind == "m" else 255)
    if kind == "m":
        v = np.where(c < 8, c * 2.0 ** -9, (1 + c % 8 / 8) * 2.0 ** (c // 8 - 7.0))
    else:
        v = (1 + c % 8 / 8) * 2.0 ** (c // 8 - 31.0)
    return torch.from_numpy(np.concatenate([[0.0], v])).cuda()


def _exact_codes(a, kind, most, u):
    """The value that is kept of a: the neighbour below, or the one above for the share u of the gap (the lowest
    binade's gaps go on below it where there is no sign, and what is not zero stays so)."""
    top = a.abs().view(-1, BLOCK).max(1)[0].cpu().numpy().astype(np.float32).astype(np.float64)
    e = np.frexp(top / most)[1]  # top is below most 2^e, and may be most 2^(e - 1)
    e = np.where(top <= most * np.ldexp(1.0, e - 1), e - 1, e)
    scale = torch.from_numpy(np.ldexp(1.0, np.clip(e, -126, 127))).to(a.device)[:, None].expand(-1, BLOCK).reshape(-1)
    table = _table(kind)
    mag = a.abs() / scale
    at = (torch.searchsorted(table, mag, right=True) - 1).clamp(max=len(table) - 2)
    low, high = table[at], table[at + 1]
    up = (mag - low) / (high - low) + u >= 1.0
    if kind == "v":
        up = torch.where(at == 0, mag > 0, up)
    return torch.where(up, high, low) * scale * torch.sign(a)


def _exact_adamw(c, s):
    t = int(s["counter"][0]) + 1
    small = c["bits"] == 8
    g = s["grad"].double() * s["grad_scale"].double()
    if small:
        each = [s[n].double().view(-1, 1).expand(-1, BLOCK).reshape(-1) for n in ("m_scale", "v_scale")]
        m0 = _table("m")[s["m"].int() & 127] * each[0] * (1 - 2 * (s["m"] > 127).double())
        v0 = _table("v")[s["v"].int()] * each[1]
        del each
    else:
        m0, v0 = s["m"].double(), s["v"].double()
    m = torch.add(BETA1 * m0, g, alpha=1 - BETA1)
    v = torch.addcmul(BETA2 * v0, g, g, value=1 - BETA2)
    del m0, v0, g
    p = (s["param"] if s["master"] is None else s["master"]).double()
    lr = float(s["lr"])
    p = p.view(-1, BLOCK) * (1 - lr * s["decays"].double())[:, None]
    step = (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)) ** 0.5 + ADAM_EPS)
    p = p.view(-1) - lr * step
    del step
    key = _mix(_mix(t) + SEED & 0xffffffff)  # whole numbers
    r = _mix(torch.arange(p.numel(), device=p.device) ^ key) if small or not c["master"] else None
    if c["master"]:
        out = [p, p]
    elif c["dtype"] == "f32":
        out = [p]
    else:
        gap = _binade(p.abs()).clamp(min=2.0 ** -126) / 128
        low = (r * 0x9e3779b1 & 0xffffffff) >> 16
        out = [torch.floor(p.abs() / gap + low.double() / 65536) * gap * torch.sign(p)]
    if small:
        m = _exact_codes(m, "m", 448.0, _share(r & 0xffff))
        v = _exact_codes(v, "v", 1.75, _share(r >> 16))
    return out + [m, v]

