"""Refusals of the operators behind the block, on the CPU: the library validates
before any HIP call, the plan's layout is host work altogether, and the binding
refuses before the library."""
import ctypes

import numpy as np
import pytest
import torch

from test_block_abi_cpu import NULL, P, lib, refuses  # noqa: F401 (lib is a fixture)
from test_block_binding_cpu import OnAnotherGpu, on, library  # noqa: F401 (library is a fixture)
from expert_grouped_gemm_top_amd import moe

F32, BF16, I32, U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8


def off(i, n):
    return ctypes.c_void_p(P(i).value + n)


def test_balance_loss(lib):  # noqa: F811
    ws = lib.moe_balance_loss_workspace_bytes(1000, 128, 3)
    assert ws > 0 and lib.moe_balance_loss_workspace_bytes(256, 128, 1) == 0
    for bad in ((0, 8, 1), (8, 0, 1), (8, 257, 1), (8, 8, 0), (8, 8, 65536)):
        assert lib.moe_balance_loss_workspace_bytes(*bad) == 0
    # T E k n_seq score alpha | logits idx offsets counts mean_p loss ws
    ok = [1000, 128, 8, 3, 0, 0.5] + [P(i) for i in range(7)] + [ws, NULL]
    refuses(lib, lib.moe_balance_loss_fwd, ok, [
        ({0: 0}, 1, "T=0"), ({1: 257}, 2, "256"), ({2: 129}, 1, "exceeds E"), ({2: 17}, 2, "16"), ({0: 1 << 28}, 2, "2^31"),
        ({3: 0}, 1, "n_seq=0"), ({3: 65536}, 2, "n_seq"), ({8: NULL}, 1, "without seq_offsets"), ({4: 2}, 1, "score"),
        ({5: float("nan")}, 1, "alpha"), ({5: float("inf")}, 1, "alpha"), ({6: NULL}, 1, "logits"), ({7: NULL}, 1, "topk_idx"),
        ({9: NULL}, 1, "counts"), ({10: NULL}, 1, "mean_p"), ({11: NULL}, 1, "loss"), ({12: NULL}, 1, "workspace"),
        ({13: ws - 1}, 3, "workspace"), ({12: off(6, 8)}, 1, "workspace must be 16-byte"), ({9: P(0)}, 1, "counts overlaps logits"),
        ({10: off(3, 16)}, 1, "counts overlaps mean_p"), ({11: P(2)}, 1, "loss overlaps seq_offsets"),
        ({12: P(4)}, 1, "workspace overlaps mean_p")])
    # T E k n_seq score alpha | logits counts offsets dloss dl_add dlogits
    ok = [1000, 128, 8, 3, 1, 0.5] + [P(i) for i in range(6)] + [NULL]
    refuses(lib, lib.moe_balance_loss_bwd, ok, [
        ({0: -1}, 1, "T=-1"), ({2: 0}, 1, "k=0"), ({3: 65536}, 2, "n_seq"), ({8: NULL}, 1, "without seq_offsets"), ({6: NULL}, 1, "logits"),
        ({7: NULL}, 1, "counts"), ({11: NULL}, 1, "dlogits"), ({11: P(0)}, 1, "dlogits overlaps logits"),
        ({11: off(4, 16)}, 1, "dlogits overlaps dl_add"), ({11: P(1)}, 1, "dlogits overlaps counts"), ({11: P(3)}, 1, "dlogits overlaps dloss")])


def test_vocab_loss(lib):  # noqa: F811
    size = lib.moe_vocab_loss_workspace_bytes
    ws = size(64, 256, 1024, 1)
    assert ws > 0 and size(1 << 24, 8, 8, 1) > 0 and size(8192, 4096, 131072, 1) < 1 << 30
    for bad in ((0, 8, 8, 1), (8, 0, 8, 1), (8, 8, -8, 1), ((1 << 24) + 1, 8, 8, 1), (8, (1 << 20) + 8, 8, 1), (8, 8, 8, 2),
                (1 << 24, 1 << 16, 8, 1)):
        assert size(*bad) == 0
    # T H V vocab dtype | x w target loss lse mean ws
    ok = [64, 256, 1024, 1000, 1] + [P(i) for i in range(7)] + [ws, NULL]
    dims = [({0: 0}, 1, "T=0"), ({0: (1 << 24) + 1}, 2, "T="), ({1: 12}, 2, "H=12"), ({2: 1028}, 2, "V=1028"), ({1: 0}, 1, "H=0"),
            ({2: (1 << 20) + 8}, 2, "exceeds"), ({0: 1 << 24, 1: 1 << 16}, 2, "too large"), ({3: 0}, 1, "vocab=0"), ({3: 1025}, 1, "vocab=1025"),
            ({4: 2}, 1, "dtype"), ({5: NULL}, 1, "x must"), ({6: NULL}, 1, "w must"), ({7: NULL}, 1, "target"), ({5: off(0, 8)}, 1, "x must be 16"),
            ({6: off(1, 2)}, 1, "w must be 16")]
    refuses(lib, lib.moe_vocab_loss_fwd, ok, dims + [
        ({8: NULL}, 1, "loss"), ({9: NULL}, 1, "lse"), ({10: NULL}, 1, "mean"), ({11: NULL}, 1, "workspace"), ({12: ws - 1}, 3, "workspace"),
        ({8: P(0)}, 1, "loss overlaps x"), ({9: off(3, 4)}, 1, "loss overlaps lse"), ({10: P(2)}, 1, "mean overlaps target"),
        ({11: off(1, 256)}, 1, "workspace overlaps w")])
    # T H V vocab dtype | x w target loss lse mean dloss | scale | dx dw ws
    ok = [64, 256, 1024, 1000, 1] + [P(i) for i in range(7)] + [1.0] + [P(i) for i in range(7, 10)] + [ws, NULL]
    refuses(lib, lib.moe_vocab_loss_bwd, ok, dims + [
        ({8: NULL}, 1, "loss"), ({9: NULL}, 1, "lse"), ({10: NULL, 11: NULL}, 1, "mean or dloss"), ({12: float("inf")}, 1, "scale"),
        ({13: NULL, 14: NULL}, 1, "no gradient"), ({13: off(7, 8)}, 1, "dx must be 16"), ({14: off(8, 8)}, 1, "dw must be 16"),
        ({13: P(0)}, 1, "dx overlaps x"), ({14: P(1)}, 1, "dw overlaps w"), ({14: off(7, 64)}, 1, "dx overlaps dw"), ({13: P(6)}, 1, "dx overlaps dloss"),
        ({15: NULL}, 1, "workspace"), ({16: ws - 1}, 3, "workspace"), ({15: P(4)}, 1, "workspace overlaps lse")])


def tensors(n, bits=32, master=False, numel=1000):
    out = (moe._AdamWEntry * n)()
    for i, e in enumerate(out):
        for j, name in enumerate(("param", "grad", "m", "v", "m_scale", "v_scale", "master")):
            if (name.endswith("scale") and bits == 32) or (name == "master" and not master):
                continue
            setattr(e, name, P(8 * i + j).value)
        e.numel, e.weight_decay = numel, 0.1
    return out


def test_adamw_plan(lib):  # noqa: F811
    size = lib.moe_adamw_plan_bytes
    assert size(0) == size(-1) == size((1 << 20) + 1) == 0 and size(3) > size(2) > 0
    plan = np.zeros(size(3), np.uint8)

    def call(t, n=3, dtype=1, bits=32, into=plan.ctypes.data, room=None):
        return lib.moe_adamw_plan(n, t, dtype, bits, into, size(3) if room is None else room)

    assert call(tensors(3)) == 0 and call(tensors(3, 8), bits=8) == 0 and call(tensors(3, 32, True)) == 0
    assert call(tensors(3, numel=0)) == 0
    for kw, status, text in ((dict(n=0), 1, "n=0"), (dict(n=(1 << 20) + 1), 2, "exceeds"), (dict(dtype=2), 1, "dtype"), (dict(bits=16), 1, "state_bits"),
                             (dict(into=NULL), 1, "plan"), (dict(room=size(3) - 1), 3, "needed")):
        assert call(tensors(3), **kw) == status and text in lib.moe_last_error().decode(), kw
    assert call(NULL) == 1 and "tensors" in lib.moe_last_error().decode()

    def refused(change, text, status=1, **kw):
        t = tensors(3, kw.get("bits", 32), kw.pop("master", False))
        change(t[1])
        assert call(t, **kw) == status and text in lib.moe_last_error().decode(), (text, lib.moe_last_error())

    refused(lambda e: setattr(e, "numel", -1), "-1 elements")
    refused(lambda e: setattr(e, "numel", 1 << 40), "elements", 2)
    for name in ("param", "grad", "m", "v"):
        refused(lambda e: setattr(e, name, None), "must not be NULL")
        refused(lambda e: setattr(e, name, getattr(e, name) + 8), f"{name} must be 16-byte")
    refused(lambda e: setattr(e, "m_scale", None), "m_scale", bits=8)
    refused(lambda e: setattr(e, "v_scale", e.v_scale + 2), "v_scale must be 4-byte", bits=8)
    refused(lambda e: setattr(e, "m_scale", P(60).value), "m_scale")
    refused(lambda e: setattr(e, "master", P(60).value), "master")
    refused(lambda e: setattr(e, "master", None), "master", master=True)
    refused(lambda e: None, "fp32 param", master=True, dtype=0)
    refused(lambda e: setattr(e, "weight_decay", -0.1), "weight_decay")
    refused(lambda e: setattr(e, "weight_decay", float("nan")), "weight_decay")
    refused(lambda e: setattr(e, "grad", e.param), "overlaps")
    refused(lambda e: setattr(e, "m", P(0).value + 1984), "overlaps")  # the last sixteen bytes of tensor 0's param


def test_the_entries_are_packed_as_the_struct():
    assert ctypes.sizeof(moe._AdamWEntry) == 72 and moe._AdamWEntry.numel.offset == 56 and moe._AdamWEntry.weight_decay.offset == 64


def test_adamw_plan_lays_out_blocks_and_chunks(lib):  # noqa: F811
    t = tensors(4)
    for e, n in zip(t, (0, 1, 4097, 256)):
        e.numel = n
    plan = np.zeros(lib.moe_adamw_plan_bytes(4), np.uint8)
    assert lib.moe_adamw_plan(4, t, 0, 32, plan.ctypes.data, plan.nbytes) == 0
    words = plan[64:].view(np.int64)
    entries, starts = words[:-5].reshape(4, -1), words[-5:]
    assert entries[:, 8].tolist() == [0, 0, 1, 18]  # blocks of 256 in front
    assert starts.tolist() == [0, 0, 1, 4, 5]       # chunks of 2048


def test_adamw_step_and_moments(lib):  # noqa: F811
    plan = np.zeros(lib.moe_adamw_plan_bytes(1), np.uint8)
    ok = [plan.ctypes.data, P(1), P(2), P(3), 0.9, 0.999, 1e-8, NULL, 0, NULL]
    assert lib.moe_adamw_step(*ok) == 1 and "not one" in lib.moe_last_error().decode()
    assert lib.moe_adamw_plan(1, tensors(1), 0, 32, plan.ctypes.data, plan.nbytes) == 0
    refuses(lib, lib.moe_adamw_step, ok, [
        ({0: NULL}, 1, "plan"), ({1: NULL}, 1, "plan_device"), ({1: off(1, 8)}, 1, "plan_device must be 16"), ({2: NULL}, 1, "counter"),
        ({3: NULL}, 1, "lr"), ({4: 1.0}, 1, "beta"), ({4: -0.1}, 1, "beta"), ({5: 1.0}, 1, "beta"), ({5: float("nan")}, 1, "beta"),
        ({6: -1e-8}, 1, "eps"), ({6: float("inf")}, 1, "eps"), ({6: 1e-40}, 2, "eps"), ({6: 1e38}, 2, "eps")])
    ok = [1000] + [P(i) for i in range(6)] + [NULL]
    refuses(lib, lib.moe_adamw_moments, ok, [({0: 0}, 1, "numel=0"), ({0: 1 << 40}, 2, "too large")] +
            [({i + 1: NULL}, 1, n) for i, n in enumerate(("m must", "v must", "m_scale", "v_scale", "m_out", "v_out"))] +
            [({1: off(0, 8)}, 1, "m must be 16"), ({5: off(4, 4)}, 1, "m_out must be 16"), ({5: P(0)}, 1, "m_out overlaps m"),
             ({6: off(4, 1600)}, 1, "m_out overlaps v_out"), ({6: P(2)}, 1, "v_out overlaps m_scale")])


T, E, K, H, V, S = 6, 8, 2, 16, 24, 3
CALLS = {
    "moe_balance_loss_fwd": dict(logits=on(T, E), topk_idx=on(T, K, dtype=I32), counts=on(S, E, dtype=I32), mean_p=on(S, E),
                                 loss=on(1), workspace=on(99, dtype=U8), seq_offsets=on(S + 1, dtype=I32)),
    "moe_balance_loss_bwd": dict(logits=on(T, E), counts=on(S, E, dtype=I32), dlogits=on(T, E), k=K, seq_offsets=on(S + 1, dtype=I32),
                                 dloss=on(1), dl_add=on(T, E)),
    "moe_vocab_loss_fwd": dict(x=on(T, H, dtype=BF16), w=on(H, V, dtype=BF16), target=on(T, dtype=I32), loss=on(T), lse=on(T), mean=on(2),
                               workspace=on(99, dtype=U8)),
    "moe_vocab_loss_bwd": dict(x=on(T, H, dtype=BF16), w=on(H, V, dtype=BF16), target=on(T, dtype=I32), loss=on(T), lse=on(T), mean=on(2),
                               dx=on(T, H, dtype=BF16), dw=on(H, V, dtype=BF16), workspace=on(99, dtype=U8), dloss=on(T)),
    "moe_adamw_moments": dict(m=on(600, dtype=U8), v=on(600, dtype=U8), m_scale=on(3), v_scale=on(3), m_out=on(600), v_out=on(600)),
}
OPTIONAL = {"workspace", "seq_offsets", "dloss", "dl_add", "mean", "dx", "dw"}
SIZES = {"logits", "x", "w", "topk_idx", "counts", "m"}  # the call's sizes come from these


@pytest.mark.parametrize("name", CALLS)
def test_the_binding_refuses_one_wrong_argument_at_a_time(library, name):  # noqa: F811
    f, ok = getattr(moe, name), CALLS[name]
    f(**ok)
    assert [c[0] for c in library.calls] == [name]
    for arg, t in ok.items():
        if not isinstance(t, torch.Tensor):
            continue
        bad = [t.as_subclass(torch.Tensor), torch.zeros_like(t).double(), t.as_subclass(OnAnotherGpu)]
        if arg not in SIZES and arg != "workspace":
            bad += [on(*t.shape, 2, dtype=t.dtype)[..., 0]] if t.numel() > 1 else []  # strides
            bad.append(on(t.shape[0] + 1, *t.shape[1:], dtype=t.dtype))
        if not (arg in OPTIONAL and name != "moe_vocab_loss_fwd"):
            bad.append(None)
        if arg == "workspace":
            bad = [bad[0], bad[2]]
        for b in bad:
            with pytest.raises(moe.MoeError):
                f(**{**ok, arg: b})
    assert len(library.calls) == 1


def test_optional_arguments_may_be_left_out(library):  # noqa: F811
    for name, ok in CALLS.items():
        n = len(library.calls)
        getattr(moe, name)(**{k: None if k in OPTIONAL and not (name == "moe_vocab_loss_fwd" and k == "mean") else v for k, v in ok.items()})
        assert len(library.calls) == n + 1


def test_a_plan_of_another_device(library, monkeypatch):  # noqa: F811
    plan = object.__new__(moe.AdamWPlan)
    plan.device_index, plan.host, plan.on_device = 1, torch.zeros(64, dtype=U8), on(64, dtype=U8)
    with pytest.raises(moe.MoeError, match="plan of device"):
        moe.moe_adamw_step(plan, on(2, dtype=I32), on(1))
    plan.device_index = 0
    moe.moe_adamw_step(plan, on(2, dtype=I32), on(1), seed=-1)
    assert library.calls[-1][1][8] == 0xffffffff
    for kw in (dict(counter=on(1, dtype=I32)), dict(lr=on(2)), dict(grad_scale=on(1, dtype=BF16)), dict(counter=on(2))):
        with pytest.raises(moe.MoeError):
            moe.moe_adamw_step(plan, **{**dict(counter=on(2, dtype=I32), lr=on(1)), **kw})


def test_launch_count_documentation_names_every_call():
    text = open(moe.PKG + "/../include/moe.h").read()
    table = text[:text.index("int64_t moe_launch_count(void);")]
    for name in ("moe_balance_loss_fwd", "moe_balance_loss_bwd", "moe_vocab_loss_fwd", "moe_vocab_loss_bwd", "moe_adamw_step", "moe_adamw_moments"):
        assert name in table
