"""The Python binding on the CPU, in front of a library that only counts its
calls: where a call makes its own tensors."""
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
