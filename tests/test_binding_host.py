"""The Python binding on the CPU, in front of a library that only counts its
calls: where a call makes its own tensors, and which tensors it refuses."""
import contextlib

import pytest
import torch

import aware_expert_routing_moe_b200 as moe


class _Library:
    """Answers every entry point: a size for the workspace queries, else 0."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 4096 if name.endswith("workspace_bytes") else 0
        return call


@pytest.fixture
def lib(monkeypatch):
    monkeypatch.setattr(moe, "_lib", _Library())
    monkeypatch.setattr(moe, "_device_of", lambda t: t.get_device(), raising=False)  # the CPU's is -1
    return moe._lib


f32 = lambda *n: torch.zeros(*n)
u8 = lambda *n: torch.zeros(*n, dtype=torch.uint8)
i16 = lambda *n: torch.zeros(*n, dtype=torch.int16)
LISTS = moe.alloc_lists(4, 8, 2, device="cpu")
B, d, E, k, F = 4, 256, 8, 2, 128
W16 = (i16(E, F, d), i16(E, F, d), i16(E, d, F))
W8 = (u8(E, F, d), f32(E, 1, 2), u8(E, F, d), f32(E, 1, 2), u8(E, d, F), f32(E, 2, 1))

# a call of every entry point that can make tensors of its own, and how many
CALLS = {
    "moe_route": (lambda s: moe.moe_route(f32(B, d), f32(E, d), None, k, stream=s), 4),
    "moe_reselect": (lambda s: moe.moe_reselect(f32(B, E), f32(B, E), k, 0, stream=s), 7),
    "moe_expert_ffn": (lambda s: moe.moe_expert_ffn(f32(B, d), *W16, LISTS, k, u8(4096), stream=s), 1),
    "moe_layer_decode": (lambda s: moe.moe_layer_decode(f32(B, d), f32(E, d), None, *W16, k, 0, stream=s), 2),
    "moe_decode_stack": (lambda s: moe.moe_decode_stack(f32(2, B, d), [(f32(E, d), None, *W16)], k, 0, stream=s), 1),
    "moe_down_channel_major": (lambda s: moe.moe_down_channel_major(W16[2], stream=s), 1),
    "moe_expert_ffn_channels": (lambda s: moe.moe_expert_ffn_channels(
        f32(B, d), W16[0], W16[1], i16(E, F, d), torch.zeros(B, k, dtype=torch.int32), f32(B, k), f32(B, k, F), 8,
        stream=s), 2),
    "moe_expert_ffn_noalloc": (lambda s: moe.moe_expert_ffn_noalloc(f32(B, d), *W16, LISTS, k, stream=s), 1),
    "moe_route_scored": (lambda s: moe.moe_route_scored(f32(B, E), k, stream=s), 8),
    "moe_quantize_blocks": (lambda s: moe.moe_quantize_blocks(f32(B, d), stream=s), 2),
    "moe_expert_gemm_blocks": (lambda s: moe.moe_expert_gemm_blocks(u8(B, d), f32(B, 2), *W8[:2], LISTS, k, stream=s), 2),
    "moe_expert_ffn_blocks": (lambda s: moe.moe_expert_ffn_blocks(f32(B, d), *W8, LISTS, k, stream=s), 2),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("handle", [0, 7])
def test_own_tensors_are_made_on_the_call_s_stream(lib, monkeypatch, name, handle):
    inside, made = [], []

    @contextlib.contextmanager
    def stream(s):
        inside.append(s)
        yield
        inside.pop()

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: ("external", h))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: ("external", 0))
    call, n = CALLS[name]
    empty, zeros = torch.empty, torch.zeros
    counting = []

    def counted(make):
        def f(*a, **kw):
            if counting and "device" in kw:  # (the test's own inputs name no device)
                made.append(list(inside))
            return make(*a, **kw)
        return f

    monkeypatch.setattr(torch, "empty", counted(empty))
    monkeypatch.setattr(torch, "zeros", counted(zeros))
    counting.append(True)
    call(handle)
    assert made == [[("external", handle)]] * n and name in lib.calls


def _good():
    """Valid arguments of the checked entry points, by name."""
    z = lambda *n, t=torch.float32: torch.zeros(*n, dtype=t)
    lists = moe.alloc_lists(B, E, k, device="cpu")
    return {
        "moe_route_scored": dict(logits=z(B, E), k=k, bias=z(E), out=(z(B, k, t=torch.int32), z(B, k)), lists=lists, ws=u8(4096)),
        "moe_quantize_blocks": dict(x=z(B, d), q=u8(B, d), scale=z(B, 2)),
        "moe_expert_gemm_blocks": dict(q=u8(B, d), scale=z(B, 2), W=u8(E, F, d), Wscale=z(E, 1, 2), lists=lists, k=k,
                                       ws=u8(4096), y=z(B * k, F)),
        "moe_expert_ffn_blocks": dict(x=z(B, d), Wgate=u8(E, F, d), Sgate=z(E, 1, 2), Wup=u8(E, F, d), Sup=z(E, 1, 2),
                                      Wdown=u8(E, d, F), Sdown=z(E, 2, 1), lists=lists, k=k, ws=u8(4096), y=z(B, d)),
    }


def test_valid_arguments_reach_the_library(lib):
    for name, kw in _good().items():
        getattr(moe, name)(**kw, stream=0)
        assert lib.calls.pop() == name
    for t in (torch.float8_e4m3fn, torch.int8):  # e4m3 as values, or as bits
        kw = _good()["moe_expert_gemm_blocks"]
        moe.moe_expert_gemm_blocks(**dict(kw, q=kw["q"].view(t), W=kw["W"].view(t)), stream=0)
    kw = _good()["moe_expert_ffn_blocks"]  # flat scales of the right size, longer lists, bf16 on either side
    moe.moe_expert_ffn_blocks(**dict(kw, Sgate=torch.zeros(E * 2), lists=moe.alloc_lists(2 * B, E, k, device="cpu"),
                                     x=kw["x"].bfloat16()), stream=0)
    assert len(lib.calls) == 3


BF, HALF, F64, I64 = torch.bfloat16, torch.float16, torch.float64, torch.int64
WRONG_TYPES = (
    [("moe_route_scored", "logits", t) for t in (BF, HALF, F64)] + [("moe_route_scored", "bias", t) for t in (BF, F64)]
    + [("moe_route_scored", "out0", I64), ("moe_route_scored", "out1", F64), ("moe_route_scored", "out0", torch.float32)]
    + [(n, l, t) for n in ("moe_route_scored", "moe_expert_gemm_blocks", "moe_expert_ffn_blocks")
       for l, t in (("lists.n_active", I64), ("lists.active", I64), ("lists.offsets", I64), ("lists.tok", I64), ("lists.w", F64))]
    + [("moe_quantize_blocks", "x", HALF), ("moe_quantize_blocks", "x", F64), ("moe_quantize_blocks", "q", torch.float8_e5m2),
       ("moe_quantize_blocks", "q", torch.float32), ("moe_quantize_blocks", "scale", F64)]
    + [("moe_expert_gemm_blocks", n, t) for n, t in (("q", BF), ("q", torch.float8_e5m2), ("scale", F64), ("W", BF),
                                                     ("W", torch.float8_e5m2), ("Wscale", F64), ("Wscale", BF), ("y", HALF))]
    + [("moe_expert_ffn_blocks", n, t) for n, t in (("x", HALF), ("Wgate", BF), ("Wup", torch.bool), ("Wdown", torch.float32),
                                                    ("Sgate", F64), ("Sup", F64), ("Sdown", BF), ("y", I64))])


def _with(kw, name, change):
    """kw with one tensor changed (`out0`: the first of out; `lists.w`)."""
    if name.startswith("out"):
        out = list(kw["out"])
        out[int(name[3:])] = change(out[int(name[3:])])
        return dict(kw, out=tuple(out))
    if "." in name:
        l = name.split(".")[1]
        return dict(kw, lists=dict(kw["lists"], **{l: change(kw["lists"][l])}))
    return dict(kw, **{name: change(kw[name])})


@pytest.mark.parametrize("entry,name,dtype", WRONG_TYPES)
def test_other_types_are_refused(lib, entry, name, dtype):
    # with as many elements as the call needs, so that only the type is wrong
    kw = _with(_good()[entry], name, lambda t: torch.zeros(t.shape, dtype=dtype))
    with pytest.raises(TypeError):
        getattr(moe, entry)(**kw, stream=0)
    assert not lib.calls


@pytest.mark.parametrize("entry,name,shape", [
    ("moe_expert_gemm_blocks", "W", (E, F, d + 16)), ("moe_expert_gemm_blocks", "W", (E, d, F)),
    ("moe_expert_gemm_blocks", "Wscale", (E, 2, 1)), ("moe_expert_gemm_blocks", "q", (B, d - 16)),
    ("moe_expert_gemm_blocks", "scale", (B, 1)), ("moe_expert_gemm_blocks", "y", (B * k - 1, F)),
    ("moe_expert_ffn_blocks", "Wup", (E, d, F)), ("moe_expert_ffn_blocks", "Wdown", (E, F, d)),
    ("moe_expert_ffn_blocks", "Wup", (E + 1, F, d)), ("moe_expert_ffn_blocks", "Wgate", (E, F, d + 16)),
    ("moe_expert_ffn_blocks", "Sup", (E, 2, 1)), ("moe_expert_ffn_blocks", "Sdown", (E, 1, 2)),
    ("moe_expert_ffn_blocks", "Sgate", (E * 2 - 1,)), ("moe_expert_ffn_blocks", "x", (B, d + 16)),
    ("moe_route_scored", "bias", (E - 1,)), ("moe_route_scored", "out0", (B, k - 1)),
    ("moe_route_scored", "lists.offsets", (E,)), ("moe_quantize_blocks", "scale", (B, 1))])
def test_other_shapes_are_refused(lib, entry, name, shape):
    kw = _with(_good()[entry], name, lambda t: torch.zeros(shape, dtype=t.dtype))
    with pytest.raises(ValueError):
        getattr(moe, entry)(**kw, stream=0)
    assert not lib.calls


class _Elsewhere(torch.Tensor):
    def get_device(self):
        return 1


@pytest.mark.parametrize("entry,name", [(e, n) for e, kw in _good().items() for n in
                                        [n for n in kw if isinstance(kw[n], torch.Tensor)]
                                        + (["out0", "out1"] if "out" in kw else [])
                                        + (["lists." + l for l in kw["lists"]] if "lists" in kw else [])])
def test_tensors_of_another_device_are_refused(lib, monkeypatch, entry, name):
    monkeypatch.setattr(moe, "_device_of", lambda t: -1, raising=False)  # the call's device
    kw = _with(_good()[entry], name, lambda t: t.as_subclass(_Elsewhere))
    first = {"moe_route_scored": "logits", "moe_quantize_blocks": "x", "moe_expert_gemm_blocks": "q", "moe_expert_ffn_blocks": "x"}
    if name == first[entry]:  # it says which device the call is on: all the others are then elsewhere
        monkeypatch.setattr(moe, "_device_of", lambda t: t.get_device(), raising=False)
    with pytest.raises(ValueError):
        getattr(moe, entry)(**kw, stream=0)
    assert not lib.calls


def test_the_call_s_device_is_the_current_one(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    with pytest.raises(ValueError):
        moe.moe_quantize_blocks(torch.zeros(4, 256).as_subclass(_Elsewhere), stream=0)
    with pytest.raises(ValueError):
        moe.moe_quantize_blocks(torch.zeros(4, 256), stream=0)
