"""Host-side checks of the scored router and the block-scaled operators that
need no GPU: workspace sizes and the status of every refused argument.

Every call with fake addresses carries at least one argument that the host
validation rejects, so none of them can reach a kernel launch."""
import os
import re

import numpy as np
import pytest
import torch

import aware_expert_routing_moe_b200 as moe
import block_cases as bc
from aware_expert_routing_moe_b200 import BlockWeights, Dims, Lists, Scoring

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, MISALIGNED, WORKSPACE = range(4)
A = 0x10000  # fake, 256-byte aligned address (never dereferenced)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from aware_expert_routing_moe_b200 import build
    build.build()
    return moe.load_library()


def test_binding_structs_and_constants_match_the_header():
    with open(os.path.join(ROOT, "include", "moe_decode.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    consts = {m.group(1): int(m.group(2)) for m in re.finditer(r"\b(MOE_[A-Z0-9_]+)\s*=\s*(\d+)", text)}
    assert moe.MOE_SCORE_SOFTMAX == consts["MOE_SCORE_SOFTMAX"] and moe.MOE_SCORE_SIGMOID == consts["MOE_SCORE_SIGMOID"]
    assert moe._DTYPES == {torch.float32: consts["MOE_F32"], torch.bfloat16: consts["MOE_BF16"]}
    assert moe.GEMM_WORKSPACE_BYTES == int(re.search(r"#define MOE_GEMM_WORKSPACE_BYTES (\d+)", text).group(1))

    def fields(tag):
        body = re.search(r"typedef struct \{([^{}]*)\}\s*" + tag + r"\s*;", text).group(1)
        return [n.strip().lstrip("*") for decl in body.split(";") if decl.strip()
                for n in re.sub(r"^(const )?\w+ ", "", decl.strip()).split(",")]
    assert fields("moe_scoring_t") == [f[0] for f in Scoring._fields_]
    assert fields("moe_block_weights_t") == [f[0] for f in BlockWeights._fields_]


def test_workspace_bytes(lib):
    n = lambda *d: int(lib.moe_blocks_workspace_bytes(Dims(*d)))
    small, big = n(1, 2048, 128, 8, 768), n(4096, 2048, 128, 8, 768)
    assert 0 < small < big and small % 256 == 0 and big % 256 == 0
    assert n(65536, 16384, 512, 16, 16384) > 1 << 32
    for bad in [(0, 2048, 128, 8, 768), (65537, 2048, 128, 8, 768), (1, 2040, 128, 8, 768), (1, 2048, 128, 8, 760),
                (1, 0, 128, 8, 768), (1, 16400, 128, 8, 768), (1, 2048, 128, 8, 16400), (1, 2048, 513, 8, 768),
                (1, 2048, 4, 8, 768), (1, 2048, 128, 17, 768), (1, 2048, 128, 0, 768)]:
        assert n(*bad) == 0, bad
    r = lambda B, E, k: int(lib.moe_route_workspace_bytes(Dims(B, 0, E, k, 0)))
    assert r(1, 256, 8) > 0 and r(65536, 512, 16) > 0
    for bad in [(0, 256, 8), (65537, 256, 8), (1, 513, 8), (1, 4, 8), (1, 256, 0), (1, 256, 17)]:
        assert r(*bad) == 0, bad
    with pytest.raises(moe.MoeError):
        moe.new_route_workspace(0, 8, 2, device="cpu")
    with pytest.raises(moe.MoeError):
        moe.new_blocks_workspace(1, 8, 8, 2, 16, device="cpu")


def _lists(**kw):
    f = dict(n_active=A, active=A, offsets=A, tok=A, w=A)
    f.update(kw)
    return Lists(*f.values())


def _route(lib, logits=A, bias=A, dims=Dims(4, 0, 64, 4, 0), rule=(1, 8, 4, 2, 1, 2.5), sel=A, w=A, lists=None, ws=A,
           n=BIG):
    return lib.moe_route_scored(logits, bias, dims, Scoring(*rule), sel, w, lists or _lists(), ws, n, None)


@pytest.mark.parametrize("change,status", [
    (dict(logits=None), INVALID), (dict(sel=None), INVALID), (dict(w=None), INVALID),
    (dict(lists=_lists(tok=None)), INVALID), (dict(lists=_lists(n_active=None)), INVALID),
    (dict(dims=Dims(0, 0, 64, 4, 0)), INVALID), (dict(dims=Dims(65537, 0, 64, 4, 0)), INVALID),
    (dict(dims=Dims(4, 0, 513, 4, 0), rule=(1, 1, 1, 1, 1, 1.0)), INVALID), (dict(dims=Dims(4, 0, 64, 17, 0)), INVALID),
    (dict(dims=Dims(4, 0, 8, 9, 0)), INVALID),
    (dict(rule=(2, 8, 4, 2, 1, 1.0)), INVALID), (dict(rule=(-1, 8, 4, 2, 1, 1.0)), INVALID),
    (dict(rule=(1, 0, 1, 1, 1, 1.0)), INVALID), (dict(rule=(1, 7, 4, 2, 1, 1.0)), INVALID),
    (dict(rule=(1, 64, 4, 1, 1, 1.0)), INVALID), (dict(rule=(1, 8, 0, 2, 1, 1.0)), INVALID),
    (dict(rule=(1, 8, 9, 2, 1, 1.0)), INVALID), (dict(rule=(1, 8, 4, 0, 1, 1.0)), INVALID),
    (dict(rule=(1, 8, 4, 3, 1, 1.0)), INVALID), (dict(rule=(1, 8, 4, 2, 2, 1.0)), INVALID),
    (dict(rule=(1, 8, 4, 2, 1, 0.0)), INVALID), (dict(rule=(1, 8, 4, 2, 1, -1.0)), INVALID),
    (dict(rule=(1, 8, 4, 2, 1, float("nan"))), INVALID), (dict(rule=(1, 8, 4, 2, 1, float("inf"))), INVALID),
    (dict(logits=A + 4), MISALIGNED), (dict(bias=A + 8), MISALIGNED), (dict(sel=A + 4), MISALIGNED),
    (dict(w=A + 2), MISALIGNED), (dict(lists=_lists(w=A + 4)), MISALIGNED), (dict(ws=A + 16), MISALIGNED),
    (dict(ws=None), WORKSPACE), (dict(n=16), WORKSPACE)])
def test_route_refusals(lib, change, status):
    assert _route(lib, **change) == status


def _quant(lib, x=A, type=0, batch=1, rows=4, cols=128, block_rows=1, q=A, s=A):
    return lib.moe_quantize_blocks(x, type, batch, rows, cols, block_rows, q, s, None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), INVALID), (dict(q=None), INVALID), (dict(s=None), INVALID), (dict(type=2), INVALID),
    (dict(type=-1), INVALID), (dict(batch=0), INVALID), (dict(rows=0), INVALID), (dict(cols=0), INVALID),
    (dict(cols=100), INVALID), (dict(cols=65552), INVALID), (dict(block_rows=64), INVALID), (dict(block_rows=0), INVALID),
    (dict(batch=1 << 20, rows=1 << 20), INVALID), (dict(batch=1 << 62, rows=1 << 62), INVALID),
    (dict(rows=(1 << 31) - 1, cols=65536), INVALID), (dict(rows=-1), INVALID),
    (dict(x=A + 8), MISALIGNED), (dict(q=A + 8), MISALIGNED), (dict(s=A + 4), MISALIGNED)])
def test_quantize_refusals(lib, change, status):
    assert _quant(lib, **change) == status


D = Dims(4, 256, 8, 2, 128)


def _gemm(lib, q=A, s=A, W=A, Ws=A, dims=D, lists=None, y=A, y_type=0, ws=A, n=BIG):
    return lib.moe_expert_gemm_blocks(q, s, W, Ws, dims, lists or _lists(), y, y_type, ws, n, None)


def _ffn(lib, x=A, x_type=0, w=None, dims=D, lists=None, y=A, y_type=1, ws=A, n=BIG):
    f = dict(Wgate=A, Sgate=A, Wup=A, Sup=A, Wdown=A, Sdown=A)
    f.update(w or {})
    return lib.moe_expert_ffn_blocks(x, x_type, BlockWeights(*f.values()), dims, lists or _lists(), y, y_type, ws, n,
                                     None)


BAD_DIMS = [Dims(0, 256, 8, 2, 128), Dims(65537, 256, 8, 2, 128), Dims(4, 250, 8, 2, 128), Dims(4, 256, 8, 2, 120),
            Dims(4, 8, 8, 2, 128), Dims(4, 16400, 8, 2, 128), Dims(4, 256, 513, 2, 128), Dims(4, 256, 8, 9, 128)]


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(s=None), INVALID), (dict(W=None), INVALID), (dict(Ws=None), INVALID),
    (dict(y=None), INVALID), (dict(y_type=2), INVALID), (dict(lists=_lists(active=None)), INVALID),
    (dict(q=A + 8), MISALIGNED), (dict(s=A + 4), MISALIGNED), (dict(W=A + 1), MISALIGNED),
    (dict(Ws=A + 4), MISALIGNED), (dict(y=A + 2), MISALIGNED), (dict(ws=A + 128), MISALIGNED),
    (dict(lists=_lists(offsets=A + 4)), MISALIGNED), (dict(ws=None), WORKSPACE), (dict(n=4095), WORKSPACE)]
    + [(dict(dims=d), INVALID) for d in BAD_DIMS])
def test_gemm_refusals(lib, change, status):
    assert _gemm(lib, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(x_type=3), INVALID), (dict(y_type=-1), INVALID),
    (dict(lists=_lists(w=None)), INVALID), (dict(x=A + 4), MISALIGNED), (dict(y=A + 4), MISALIGNED),
    (dict(ws=A + 64), MISALIGNED), (dict(ws=None), WORKSPACE), (dict(n=4096), WORKSPACE)]
    + [(dict(w={n: None}), INVALID) for n in ("Wgate", "Sgate", "Wup", "Sup", "Wdown", "Sdown")]
    + [(dict(w={n: A + 8}), MISALIGNED) for n in ("Wgate", "Sgate", "Wup", "Sup", "Wdown", "Sdown")]
    + [(dict(dims=d), INVALID) for d in BAD_DIMS])
def test_ffn_refusals(lib, change, status):
    assert _ffn(lib, **change) == status


def test_binding_refuses_other_types_and_strides(lib):
    with pytest.raises(TypeError):
        moe.moe_quantize_blocks(torch.zeros(4, 128, dtype=torch.float16))
    with pytest.raises(ValueError):
        moe.moe_quantize_blocks(torch.zeros(4, 256)[:, ::2], q=torch.zeros(4, 128, dtype=torch.uint8),
                                scale=torch.zeros(4, 1), stream=0)


def test_binding_refuses_short_buffers_and_host_tensors(lib):
    z = lambda *n, t=torch.uint8: torch.zeros(*n, dtype=t)
    f = lambda *n: torch.zeros(*n)
    lists = moe.alloc_lists(4, 8, 2, device="cpu")
    ok = dict(x=f(4, 256), Wgate=z(8, 128, 256), Sgate=f(8, 1, 2), Wup=z(8, 128, 256), Sup=f(8, 1, 2),
              Wdown=z(8, 256, 128), Sdown=f(8, 2, 1), lists=lists, k=2, ws=z(1 << 20), y=f(4, 256), stream=0)
    for name, short in (("Sgate", f(8, 1, 1)), ("Wup", z(8, 127, 256)), ("Wdown", z(8, 255, 128)), ("Sdown", f(15)),
                        ("y", f(3, 256)), ("lists", dict(lists, tok=lists["tok"][:7])),
                        ("lists", dict(lists, offsets=lists["offsets"][:8]))):
        with pytest.raises(ValueError):
            moe.moe_expert_ffn_blocks(**dict(ok, **{name: short}))
    with pytest.raises(ValueError):
        moe.moe_expert_gemm_blocks(z(4, 256), f(4, 1), z(8, 128, 256), f(8, 1, 2), lists, 2, ws=z(4096), y=f(8, 128), stream=0)
    with pytest.raises(ValueError):
        moe.moe_quantize_blocks(f(4, 256), q=z(4, 255), scale=f(4, 2), stream=0)
    with pytest.raises(ValueError):
        moe.moe_route_scored(f(4, 8), 2, bias=f(7), out=(z(4, 2, t=torch.int32), f(4, 2)), lists=lists, ws=z(4096), stream=0)
    # without a stream of the caller's, tensors have to be on the current device
    with pytest.raises(ValueError):
        moe.moe_quantize_blocks(f(4, 256))


# ------------------------------------------- the restatements themselves --
def test_e4m3_restatement():
    b = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(b).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(np.nan_to_num(bc.e4m3_decode(b), nan=1e9), np.nan_to_num(want, nan=1e9))
    x = np.random.default_rng(0).uniform(-448, 448, 4096).astype(np.float32)
    x = np.concatenate([x, x * np.float32(1e-3), x * np.float32(1e-5)])
    assert np.array_equal(bc.e4m3_round(x), torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy())


def test_route_restatement_by_hand():
    l = np.log(np.array([[1.0, 3.0, 2.0, 2.0]]))
    sel, w = bc.route(l, 2, False)
    assert sel.tolist() == [[1, 2]] and np.allclose(w, [[0.6, 0.4]])
    sel, w = bc.route(l, 2, False, bias=[0.5, 0, 0, 0], renorm=False, scale=2.0)
    assert sel.tolist() == [[0, 1]] and np.allclose(w, [[0.25, 0.75]])
    sel, _ = bc.route(l, 2, False, groups=2, top_groups=1, best=2)  # both groups sum to 1/2
    assert sel.tolist() == [[1, 0]]
    L = bc.lists_of(np.array([[1, -1], [0, 1]]), np.array([[1.0, 0], [2.0, 3.0]]), 3)
    assert L["n_active"] == 2 and L["active"].tolist() == [0, 1, -1] and L["offsets"].tolist() == [0, 1, 3, 3]
    assert L["tok"].tolist() == [1, 0, 1, -1] and L["w"].tolist() == [2.0, 1.0, 3.0, 0.0]
