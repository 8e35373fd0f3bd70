"""The binding's checks of the operators around the expert path, one wrong argument
at a time: every call below is valid but for that argument, and is refused with a
message that names it, before the library is reached (a stand-in that counts).
Tensors are host memory that says it is on GPU 0."""
import pytest
import torch

from expert_grouped_gemm_top_amd import moe

T, E, K, H, I, O = 6, 8, 2, 16, 24, 40  # noqa: E741
F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32


class OnGpu(torch.Tensor):
    index = 0

    @property
    def device(self):
        return torch.device("cuda", self.index)

    @property
    def is_cuda(self):
        return True

    def get_device(self):
        return self.index


class OnAnotherGpu(OnGpu):
    index = 1


def on(*shape, dtype=F32, cls=OnGpu):
    return torch.zeros(*shape, dtype=dtype).as_subclass(cls)


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    fake = Library()
    monkeypatch.setattr(moe, "_lib", fake)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 77, raising=False)
    return fake


SPACE = on(256, dtype=torch.uint8)
CALLS = {
    "moe_route_scored": dict(logits=on(T, E), bias=on(E), topk_idx=on(T, K, dtype=I32), topk_w=on(T, K), k=K),
    "moe_route_scored_bwd": dict(logits=on(T, E), topk_idx=on(T, K, dtype=I32), dg=on(T, K), dlogits=on(T, E)),
    "moe_router_bwd_dlogits": dict(x=on(T, H, dtype=BF16), w_r=on(H, E, dtype=BF16), dlogits=on(T, E),
                                   dw_r=on(H, E, dtype=BF16), dx=on(T, H, dtype=BF16), accumulate=True, workspace=SPACE),
    "moe_layernorm_fwd": dict(x=on(T, H, dtype=BF16), gamma=on(H, dtype=BF16), beta=on(H, dtype=BF16),
                              y=on(T, H, dtype=BF16), mean=on(T), rstd=on(T)),
    "moe_layernorm_bwd": dict(x=on(T, H, dtype=BF16), gamma=on(H, dtype=BF16), mean=on(T), rstd=on(T),
                              dy=on(T, H, dtype=BF16), dx=on(T, H, dtype=BF16), dgamma=on(H, dtype=BF16),
                              dbeta=on(H, dtype=BF16), workspace=SPACE, dx_add=on(T, H, dtype=BF16)),
    "moe_linear_fwd": dict(x=on(T, I, dtype=BF16), w=on(I, O, dtype=BF16), bias=on(O, dtype=BF16), y=on(T, O, dtype=BF16),
                           mul=on(T, O, dtype=BF16), residual=on(T, O, dtype=BF16), z_save=on(T, O, dtype=BF16),
                           workspace=SPACE),
    "moe_linear_bwd": dict(x=on(T, I, dtype=BF16), w=on(I, O, dtype=BF16), dy=on(T, O, dtype=BF16), dz=on(T, O, dtype=BF16),
                           dx=on(T, I, dtype=BF16), dw=on(I, O, dtype=BF16), dbias=on(O, dtype=BF16), act=4,
                           z=on(T, O, dtype=BF16), mul=on(T, O, dtype=BF16), dmul=on(T, O, dtype=BF16),
                           dx_add=on(T, I, dtype=BF16), workspace=SPACE),
}
OPTIONAL = {"bias", "beta", "mean", "rstd", "mul", "residual", "z_save", "z", "dz", "dmul", "dx_add", "dbeta", "dbias",
            "workspace"}
ALSO_OPTIONAL = {"moe_linear_bwd": {"dx", "dw"}}
REQUIRED = {"moe_layernorm_bwd": {"mean", "rstd"}}
SIZES = {"logits", "x", "w", "w_r"}  # the call's sizes come from these
TENSORS = [(f, n) for f, a in CALLS.items() for n, v in a.items() if isinstance(v, torch.Tensor)]


def may_be_none(f, name):
    return (name in OPTIONAL or name in ALSO_OPTIONAL.get(f, ())) and name not in REQUIRED.get(f, ())


@pytest.mark.parametrize("f", CALLS)
def test_the_valid_call_reaches_the_library(library, f):
    getattr(moe, f)(**CALLS[f])
    assert [n for n, _ in library.calls] == [f]
    args = library.calls[0][1]
    assert args[-1] == 77
    for v in CALLS[f].values():
        assert not isinstance(v, torch.Tensor) or v.data_ptr() in args


def refused(library, f, message, **changed):
    with pytest.raises(moe.MoeError, match=message):
        getattr(moe, f)(**{**CALLS[f], **changed})
    assert not library.calls


@pytest.mark.parametrize("f,name", TENSORS)
def test_one_wrong_tensor(library, f, name):
    t = CALLS[f][name]
    refused(library, f, f"{name} must be a GPU tensor", **{name: torch.zeros(t.shape, dtype=t.dtype)})
    if name not in SIZES | {"workspace", "topk_idx"}:
        refused(library, f, f"{name} must be a GPU tensor", **{name: t.tolist()})
    wide = on(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype)[..., ::2]
    refused(library, f, f"{name} must be contiguous", **{name: wide})
    refused(library, f, f"{name} is on cuda:1 in a call on the current device cuda:0",
            **{name: on(*t.shape, dtype=t.dtype, cls=OnAnotherGpu)})
    if may_be_none(f, name):
        getattr(moe, f)(**{**CALLS[f], name: None})
        assert len(library.calls) == 1 and t.data_ptr() not in library.calls.pop()[1]
    else:
        refused(library, f, f"{name} (is required|must be a GPU tensor)", **{name: None})
    if name == "workspace":  # of any type and shape
        return
    other = torch.float64 if name in ("x", "logits") else (F32 if t.dtype != F32 else BF16)
    refused(library, f, "unsupported dtype" if name == "x" else f"{name} must be torch", **{name: on(*t.shape, dtype=other)})
    if name not in SIZES:
        for shape in ((t.shape[0] + 1, *t.shape[1:]), (*t.shape[:-1], t.shape[-1] - 1), (*t.shape, 1), (t.numel() * 2,)):
            if not (name == "topk_idx" and f == "moe_route_scored_bwd"):
                refused(library, f, f"{name} has shape", **{name: on(*shape, dtype=t.dtype)})


@pytest.mark.parametrize("f,name", [(f, n) for f, n in TENSORS if n in SIZES])
def test_sizes_that_do_not_fit_the_others(library, f, name):
    """Another size is one of the whole call: some other tensor no longer fits, or the shape is no matrix."""
    t = CALLS[f][name]
    refused(library, f, "has shape", **{name: on(t.shape[0] + 1, t.shape[1], dtype=t.dtype)})
    refused(library, f, "has shape", **{name: on(t.shape[0], t.shape[1] + 1, dtype=t.dtype)})
    for shape in ((t.numel(),), (1, *t.shape), (0, t.shape[1]), (t.shape[0], 0)):
        refused(library, f, f"{name} must be a matrix", **{name: on(*shape, dtype=t.dtype)})


def test_lists_of_another_length(library):
    refused(library, "moe_route_scored", "topk_idx has shape", k=K + 1)
    refused(library, "moe_route_scored_bwd", "dg has shape", topk_idx=on(T, K + 1, dtype=I32))
    refused(library, "moe_route_scored_bwd", "topk_idx has shape", topk_idx=on(T + 1, K, dtype=I32))
    refused(library, "moe_route_scored_bwd", "topk_idx must be a matrix", topk_idx=on(T * K, dtype=I32))


@pytest.mark.parametrize("f", CALLS)
def test_streams(library, f):
    class Stream:
        cuda_stream, device_index = 123, 0

    getattr(moe, f)(**CALLS[f], stream=Stream())
    assert library.calls.pop()[1][-1] == 123
    getattr(moe, f)(**CALLS[f], stream=45)
    assert library.calls.pop()[1][-1] == 45
    Stream.device_index = 1
    refused(library, f, "a stream of device cuda:1 in a call on the current device cuda:0", stream=Stream())
