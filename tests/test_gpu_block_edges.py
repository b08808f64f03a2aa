"""The block-scaled operators where they can go wrong: infinities and NaN,
wide quantisation of ragged columns, mixed types, re-selected lists, damaged
lists of large tiles, calls on another stream without a workspace, and one
workspace for all entry points in turn."""
import numpy as np
import pytest
import torch

import aware_expert_routing_moe_b200 as moe
import block_cases as bc
from test_gpu_blocks import BF16, F32, _check_ffn, _check_quantized, _choice, _cuda, _ffn_setup, _lists, _values, _weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    moe.load_library()
    yield
    torch.cuda.synchronize()


# ---------------------------------------------------------- quantisation --
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", [(2047, 144), (2048, 16), (2049, 1040), (2500, 2064), (2048, 4112)])
def test_quantize_many_rows(dtype, rows, cols):
    g = torch.Generator().manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp(3 * torch.randn(rows, 1, generator=g))
    _check_quantized(x.to(dtype).cuda(), 1)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols,block_rows", [(7, 400, 1), (2100, 1040, 1), (300, 272, 128)])
def test_infinities_and_nan_become_nan(dtype, rows, cols, block_rows):
    # and the finite values of their blocks are rounded as if they were zeros
    rng = np.random.default_rng([rows, cols])
    x = torch.from_numpy(rng.standard_normal((rows, cols)).astype(np.float32)).to(dtype).float().numpy()
    bad = rng.random((rows, cols)) < 0.002
    bad[0, :130] = True                  # whole blocks of a row
    bad[1, 5] = bad[2, 140] = bad[3, cols - 1] = True
    bad[4] = False
    kind = rng.integers(0, 3, (rows, cols))
    kind[1, 5], kind[2, 140], kind[3, cols - 1] = 0, 1, 2
    dirty = np.where(bad, np.choose(kind, [np.float32(np.inf), np.float32(-np.inf), np.float32(np.nan)]), x)
    q, s = moe.moe_quantize_blocks(_cuda(dirty.astype(np.float32)).to(dtype), block_rows)
    rq, rs = bc.quantize(np.where(bad, 0.0, x), block_rows)
    got = _values(q)
    assert np.array_equal(np.isnan(got), bad)
    assert np.array_equal(np.where(bad, 0.0, got), np.where(bad, 0.0, rq))
    assert np.array_equal(s.double().cpu().numpy(), rs)


# ------------------------------------------------------ products and FFN --
def test_product_keeps_nan_in_its_rows():
    rng = np.random.default_rng(3)
    for B, E, k in ((20, 6, 2), (300, 2, 1)):  # tiles of 16 and of 128 entries
        d, F = 272, 400
        sel, w = _choice(rng, B, E, k)
        L, dev = _lists(sel, w, E)
        x = torch.from_numpy(rng.standard_normal((B, d)).astype(np.float32)).cuda()
        bad = [1, 7, B - 1]
        dirty = x.clone()
        dirty[1, 3], dirty[7, 271], dirty[B - 1, 130] = float("inf"), float("nan"), float("-inf")
        Wq, Ws, _ = _weights(rng, E, F, d)
        ys = []
        for v in (x, dirty):
            q, s = moe.moe_quantize_blocks(v)
            ys.append(moe.moe_expert_gemm_blocks(q, s, Wq, Ws, dev, k, y_dtype=F32)[:L["offsets"][-1]])
        hit = torch.from_numpy(np.isin(L["tok"][:L["offsets"][-1]], bad)).cuda()
        assert torch.isnan(ys[1][hit]).all() and torch.equal(ys[1][~hit], ys[0][~hit])


SIZES = [(20, 272, 6, 3, 400), (150, 512, 4, 3, 256), (40, 256, 40, 3, 128)]  # tiles of 16, 128 and 16 entries


@pytest.mark.parametrize("B,d,E,k,F", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_ffn_of_a_row_that_is_not_finite_is_nan(B, d, E, k, F, dtype, value):
    L, dev, x, args, vals = _ffn_setup(B, d, E, k, F, dtype)
    clean = moe.moe_expert_ffn_blocks(x, *args, dev, k)
    dirty = x.clone()
    dirty[3, d - 1] = dirty[B - 1, 0] = dirty[B // 2, 140] = value
    y = moe.moe_expert_ffn_blocks(dirty, *args, dev, k)
    bad = torch.zeros(B, dtype=torch.bool, device="cuda")
    bad[[3, B - 1, B // 2]] = True
    assert torch.isnan(y[bad]).all() and torch.equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("B,d,E,k,F", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_ffn_whose_h_overflows_is_nan(B, d, E, k, F, dtype):
    # gate and up are about 1e32 each, their product is past fp32
    L, dev, x, args, vals = _ffn_setup(B, d, E, k, F, dtype)
    clean = moe.moe_expert_ffn_blocks(x, *args, dev, k)
    dirty = x.clone()
    dirty[5] *= 1e30
    y = moe.moe_expert_ffn_blocks(dirty, *args, dev, k)
    other = torch.arange(B, device="cuda") != 5
    assert torch.isnan(y[5]).all() and torch.equal(y[other], clean[other])


@pytest.mark.parametrize("x_dtype,y_dtype", [(BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("B,d,E,k,F", [(1, 256, 4, 2, 128), (17, 512, 8, 4, 256), (260, 272, 2, 2, 144), (3, 16, 2, 1, 16)])
def test_ffn_of_one_type_into_the_other(B, d, E, k, F, x_dtype, y_dtype):
    L, dev, x, args, vals = _ffn_setup(B, d, E, k, F, x_dtype)
    y = moe.moe_expert_ffn_blocks(x, *args, dev, k, y_dtype=y_dtype)
    assert y.dtype == y_dtype
    _check_ffn(y, x, L, vals)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_ffn_of_a_long_padded_batch(dtype):
    # rows copied to their entries by the wide quantisation, some skipped
    L, dev, x, args, vals = _ffn_setup(900, 272, 6, 3, 144, dtype, empty=0.2)
    assert L["offsets"][-1] < 2700
    ws = moe.new_blocks_workspace(900, 272, 6, 3, 144)
    y = moe.moe_expert_ffn_blocks(x, *args, dev, 3, ws=ws)
    assert moe.moe_check_error(ws) == 0
    _check_ffn(y, x, L, vals)


@pytest.mark.parametrize("B,mode,kw", [(8, moe.MOE_RESELECT_OEA, dict(k0=2)), (64, moe.MOE_RESELECT_XSHARE, dict(budget=8)),
                                       (128, moe.MOE_RESELECT_XSHARE, dict(budget=6)),
                                       (128, moe.MOE_RESELECT_XSHARE_HIER, dict(budget=16, group=4)),
                                       (100, moe.MOE_RESELECT_AFFINITY, {}), (256, moe.MOE_RESELECT_NONE, {})])
def test_lists_of_the_reselection_rules(B, mode, kw):
    d, E, k, F = 256, 64, 4, 128
    rng = np.random.default_rng([21, B])
    x = torch.from_numpy(rng.standard_normal((B, d)).astype(np.float32)).cuda()
    Wg = torch.from_numpy((rng.standard_normal((E, d)) * 0.1).astype(np.float32)).cuda()
    logits, probs, _, _ = moe.moe_route(x, Wg, None, k)
    _, _, dev = moe.moe_reselect(logits, probs, k, mode, **kw)
    L = {n: v.cpu().numpy() for n, v in dev.items()}
    L["n_active"] = int(L["n_active"][0])
    mats = [_weights(rng, E, F, d), _weights(rng, E, F, d), _weights(rng, E, d, F)]
    ws = moe.new_blocks_workspace(B, d, E, k, F)
    y = moe.moe_expert_ffn_blocks(x, *[t for m in mats for t in m[:2]], dev, k, ws=ws)
    assert moe.moe_check_error(ws) == 0
    _check_ffn(y, x, L, [m[2] for m in mats])


# --------------------------------------------------------- damaged lists --
@pytest.mark.parametrize("B,d,E,k,F", SIZES[:2])
@pytest.mark.parametrize("field,value", [("n_active", -1), ("n_active", 99), ("n_active", 2 ** 31 - 1), ("active", 6),
                                         ("active", -2), ("active", -2 ** 31), ("offsets", 10 ** 6), ("offsets", -3),
                                         ("tok", 150), ("tok", -1), ("tok", 2 ** 31 - 1), ("tok", -2 ** 31)])
def test_damaged_lists_touch_nothing_else(B, d, E, k, F, field, value):
    L, dev, x, args, vals = _ffn_setup(B, d, E, k, F, BF16)
    dev = {n: v.clone() for n, v in dev.items()}
    dev[field][1 if field == "offsets" else 0] = value
    ws, gws = moe.new_blocks_workspace(B, d, E, k, F), moe.new_gemm_workspace()
    guard = 16
    buf = torch.full((B + 2 * guard, d), 3.0, dtype=BF16, device="cuda")
    moe.moe_expert_ffn_blocks(x, *args, dev, k, ws=ws, y=buf[guard:guard + B])
    assert moe.moe_check_error(ws) == 6
    assert torch.all(buf[:guard] == 3) and torch.all(buf[guard + B:] == 3)
    gbuf = torch.full((B * k + 2 * guard, F), 5.0, dtype=BF16, device="cuda")
    q, s = moe.moe_quantize_blocks(x)
    moe.moe_expert_gemm_blocks(q, s, args[0], args[1], dev, k, ws=gws, y=gbuf[guard:guard + B * k])
    assert moe.moe_check_error(gws) == 6
    assert torch.all(gbuf[:guard] == 5) and torch.all(gbuf[guard + B * k:] == 5)
    if field != "tok":  # runs as an empty call
        assert torch.all(buf[guard:guard + B] == 0) and torch.all(gbuf == 5)


# ------------------------------------------- streams, workspaces, limits --
def _held(side):
    """Keeps the stream busy for some 50 ms."""
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)


def _litter():
    """Writes over what the current stream's allocator hands out."""
    return [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in
            [512, 1024, 4096, 4352, 16384] * 8 + [1 << 16, 1 << 18, 1 << 20, 1 << 21, 1 << 22, 1 << 24]]


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("B,E", [(20, 6), (150, 4)])
def test_calls_on_another_stream_make_their_buffers_there(B, E, raw):
    # the workspace and the outputs belong to the call's stream: what the
    # current stream allocates and writes meanwhile is other memory
    d, k, F = 256, 3, 256
    L, dev, x, args, vals = _ffn_setup(B, d, E, k, F, BF16)
    logits = torch.from_numpy(np.random.default_rng(B).standard_normal((B * 10, 32)).astype(np.float32)).cuda()
    q, s = moe.moe_quantize_blocks(x)
    n = L["offsets"][-1]
    want = (moe.moe_expert_ffn_blocks(x, *args, dev, k), moe.moe_expert_gemm_blocks(q, s, args[0], args[1], dev, k)[:n], q, s,
            *moe.moe_route_scored(logits, 4)[:2])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    to = side.cuda_stream if raw else side
    for call in range(4):
        _held(side)
        if call == 0:
            got = [moe.moe_expert_ffn_blocks(x, *args, dev, k, stream=to)]
        elif call == 1:
            got = [moe.moe_expert_gemm_blocks(q, s, args[0], args[1], dev, k, stream=to)]
        elif call == 2:
            got = list(moe.moe_quantize_blocks(x, stream=to))
        else:
            got = list(moe.moe_route_scored(logits, 4, stream=to)[:2])
        litter = _litter()
        del litter
        litter = _litter()
        side.synchronize()
        torch.cuda.synchronize()
        for g, w in zip(got, ([want[0]], [want[1]], want[2:4], want[4:])[call]):
            g = g[:n] if call == 1 else g
            assert torch.equal(g.view(torch.uint8), w.view(torch.uint8)), call


def test_one_workspace_serves_the_layer_the_router_and_the_experts_in_turn():
    B, d, E, k, F = 40, 256, 32, 4, 128
    rng = np.random.default_rng(31)
    t = lambda *n: torch.from_numpy((rng.standard_normal(n) * 0.05).astype(np.float32)).cuda()
    x, Wg = t(B, d) * 20, t(E, d)
    bf = [m.bfloat16().view(torch.int16) for m in (t(E, F, d), t(E, F, d), t(E, d, F))]
    q8 = [u for m in (t(E, F, d), t(E, F, d), t(E, d, F)) for u in moe.moe_quantize_blocks(m, 128)]
    logits = t(5000, E) * 20
    ws = torch.zeros(max(moe.moe_workspace_bytes(B, d, E, k, F), moe.new_route_workspace(5000, E, k).numel(),
                         moe.new_blocks_workspace(B, d, E, k, F).numel()), dtype=torch.uint8, device="cuda")
    first = None
    for _ in range(3):
        sel = torch.empty(B, k, dtype=torch.int32, device="cuda")
        y = moe.moe_layer_decode(x, Wg, None, *bf, k, moe.MOE_RESELECT_OEA, k0=2, ws=ws, sel_idx=sel)
        assert moe.moe_check_error(ws) == 0
        lsel, lw, _ = moe.moe_route_scored(logits, k, ws=ws)
        small, _, lists = moe.moe_route_scored(logits[:B].contiguous(), k, ws=ws)
        y8 = moe.moe_expert_ffn_blocks(x, *q8, lists, k, ws=ws)
        assert moe.moe_check_error(ws) == 0
        got = [y, sel, lsel, lw, small, y8]
        first = first or [g.clone() for g in got]
        assert float((y - first[0]).norm() / y.norm()) < 1e-5  # the layer's fp32 atomics add in any order
        for g, w in zip(got[1:], first[1:]):
            assert torch.equal(g, w)


@pytest.mark.parametrize("limit", [2 ** 62, 2 ** 63, 2 ** 64 - 1])
def test_the_longest_wait_limits(limit):
    L, dev, x, args, vals = _ffn_setup(150, 512, 4, 3, 256, BF16)
    ws, gws = moe.new_blocks_workspace(150, 512, 4, 3, 256), moe.new_gemm_workspace()
    q, s = moe.moe_quantize_blocks(x)
    try:
        moe.moe_set_wait_limit_ns(limit)
        y = moe.moe_expert_ffn_blocks(x, *args, dev, 3, ws=ws)
        moe.moe_expert_gemm_blocks(q, s, args[0], args[1], dev, 3, ws=gws)
        assert moe.moe_check_error(ws) == 0 and moe.moe_check_error(gws) == 0
    finally:
        moe.moe_set_wait_limit_ns(0)
    _check_ffn(y, x, L, vals)


@pytest.mark.parametrize("B,d,E,k,F", SIZES[:2])
def test_a_tile_counter_below_zero_is_reported(B, d, E, k, F):
    # as in a workspace that was never zero-filled: nothing is written out of
    # place, and the last CTA puts the counter right
    L, dev, x, args, vals = _ffn_setup(B, d, E, k, F, BF16)
    ws, guard = moe.new_blocks_workspace(B, d, E, k, F), 16
    buf = torch.full((B + 2 * guard, d), 3.0, dtype=BF16, device="cuda")
    ws.view(torch.int32)[1] = -5000
    moe.moe_expert_ffn_blocks(x, *args, dev, k, ws=ws, y=buf[guard:guard + B])
    assert moe.moe_check_error(ws) == 6
    assert torch.all(buf[:guard] == 3) and torch.all(buf[guard + B:] == 3)
    y = moe.moe_expert_ffn_blocks(x, *args, dev, k, ws=ws)
    assert moe.moe_check_error(ws) == 0
    _check_ffn(y, x, L, vals)


@pytest.mark.parametrize("B", [12, 300])
def test_calls_captured_without_a_workspace(B):
    # the graph holds the workspaces and their zero-fills
    d, E, k, F = 256, 8, 2, 128
    L, dev, x, args, vals = _ffn_setup(B, d, E, k, F, BF16)
    logits = torch.from_numpy(np.random.default_rng(B).standard_normal((B, E)).astype(np.float32)).cuda()

    def chain():
        sel, w, lists = moe.moe_route_scored(logits, k)
        q, s = moe.moe_quantize_blocks(x)
        return sel, w, moe.moe_expert_gemm_blocks(q, s, args[0], args[1], lists, k), moe.moe_expert_ffn_blocks(x, *args, lists, k)

    want = [t.clone() for t in chain()]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = chain()
    for _ in range(3):
        for t in got:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_the_default_stream_by_its_handle():
    L, dev, x, args, vals = _ffn_setup(150, 256, 4, 3, 256, BF16)
    want = moe.moe_expert_ffn_blocks(x, *args, dev, 3)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):  # the call runs on the default stream all the same
        y = moe.moe_expert_ffn_blocks(x, *args, dev, 3, stream=0)
        litter = _litter()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_activations_may_be_overwritten_by_the_result():
    for B, d, E, k, F in SIZES:
        L, dev, x, args, vals = _ffn_setup(B, d, E, k, F, BF16)
        want = moe.moe_expert_ffn_blocks(x, *args, dev, k)
        assert torch.equal(moe.moe_expert_ffn_blocks(x, *args, dev, k, y=x), want)


@pytest.mark.parametrize("B", [5, 200])  # tiles of 16 and of 128 entries
def test_product_of_the_largest_matrix(B):
    d = F = 16384
    g = torch.Generator(device="cuda").manual_seed(1)
    W = torch.randint(0, 256, (1, F, d), device="cuda", dtype=torch.uint8, generator=g)
    W = torch.where((W & 0x7F) == 0x7F, torch.full_like(W, 0x30), W)
    S = torch.rand(1, F // 128, d // 128, device="cuda", generator=g) * 0.02 + 0.01
    q, s = moe.moe_quantize_blocks(torch.randn(B, d, device="cuda", generator=g))
    lists = {"n_active": _cuda(np.array([1, 0, 0, 0], np.int32)), "active": _cuda(np.zeros(1, np.int32)),
             "offsets": _cuda(np.array([0, B], np.int32)), "tok": _cuda(np.arange(B, dtype=np.int32)),
             "w": torch.ones(B, device="cuda")}
    y = moe.moe_expert_gemm_blocks(q, s, W, S, lists, 1, y_dtype=F32)
    x = _values(q) * bc.spread(s.cpu().numpy().astype(np.float64), B, d, 1)
    rows = np.unique(np.r_[0, 127, 128, 255, 256, F - 257, F - 128, F - 1, np.random.default_rng(2).integers(0, F, 40)])
    at = torch.from_numpy(rows).cuda()
    w = bc.e4m3_decode(W[0][at].cpu().numpy()) * np.repeat(S[0][at // 128].cpu().numpy().astype(np.float64), 128, 1)
    ref = x @ w.T
    got = y[:, at].double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= bc.sum_bound(d, np.abs(x) @ np.abs(w).T) + bc.HALF_STEP["f32"] * np.abs(ref))


@pytest.mark.parametrize("B", [6, 40, 100])
def test_one_workspace_serves_every_entry_point_in_any_order(B):
    d, E, k, F = 256, 32, 4, 128
    rng = np.random.default_rng([41, B])
    t = lambda *n: torch.from_numpy((rng.standard_normal(n) * 0.05).astype(np.float32)).cuda()
    x, Wg = t(B, d) * 20, t(E, d)
    bf = [m.bfloat16().view(torch.int16) for m in (t(E, F, d), t(E, F, d), t(E, d, F))]
    q8 = [u for m in (t(E, F, d), t(E, F, d), t(E, d, F)) for u in moe.moe_quantize_blocks(m, 128)]
    logits, many = t(B, E) * 20, t(3000, E) * 20
    lists = moe.moe_route_scored(logits, k)[2]
    q, s = moe.moe_quantize_blocks(x)
    xs = torch.zeros(3, B, d, device="cuda")

    def stack(ws):
        xs[0] = x
        return moe.moe_decode_stack(xs, [(Wg, None, *bf)] * 2, k, moe.MOE_RESELECT_XSHARE, budget=12, ws=ws)[1].clone()

    calls = {
        "layer": lambda ws: moe.moe_layer_decode(x, Wg, None, *bf, k, moe.MOE_RESELECT_AFFINITY, ws=ws),
        "stack": stack,
        "ffn": lambda ws: moe.moe_expert_ffn(x, *bf, lists, k, ws),
        "route": lambda ws: moe.moe_route_scored(many, k, ws=ws)[1],
        "route_few": lambda ws: moe.moe_route_scored(logits, k, ws=ws)[1],
        "gemm": lambda ws: moe.moe_expert_gemm_blocks(q, s, *q8[:2], lists, k, ws=ws),
        "ffn8": lambda ws: moe.moe_expert_ffn_blocks(x, *q8, lists, k, ws=ws),
    }
    n = max(moe.moe_workspace_bytes(B, d, E, k, F), moe.new_route_workspace(3000, E, k).numel(),
            moe.new_blocks_workspace(B, d, E, k, F).numel(), 4096)
    want = {name: call(torch.zeros(n, dtype=torch.uint8, device="cuda")) for name, call in calls.items()}
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    for name in [rng.permutation(list(calls)) for _ in range(12)]:
        for c in name:
            y = calls[c](ws)
            assert moe.moe_check_error(ws) == 0, c
            # the bf16 paths add with fp32 atomics, in any order: some tens of
            # additions, 2^-24 each
            assert float((y.float() - want[c].float()).norm() / want[c].float().norm()) < 1e-5, c
