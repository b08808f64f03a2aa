"""GPU parity of the block-scaled 8-bit operators (quantisation, grouped
product, expert FFN) against 64-bit restatements on the CPU, and their
behaviour on ragged sizes, short lists, streams, graphs and bad lists."""
import numpy as np
import pytest
import torch

import aware_expert_routing_moe_b200 as moe
import block_cases as bc

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    moe.load_library()
    yield
    torch.cuda.synchronize()


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _values(q):
    return bc.e4m3_decode(q.view(torch.uint8).cpu().numpy())


# ---------------------------------------------------------- quantisation --
def _check_quantized(x, block_rows):
    q, s = moe.moe_quantize_blocks(x, block_rows)
    xs = x.double().cpu().numpy().reshape(-1, *x.shape[-2:])
    qs = _values(q).reshape(xs.shape)
    ss = s.cpu().numpy().astype(np.float64).reshape(xs.shape[0], -1, s.shape[-1])
    for b in range(xs.shape[0]):
        rq, rs = bc.quantize(xs[b], block_rows)
        assert np.array_equal(ss[b], rs)
        assert np.array_equal(qs[b], rq)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 128), (3, 144), (65, 2064), (2, 65536)])
def test_quantize_rows(dtype, rows, cols):
    g = torch.Generator().manual_seed(rows * cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp(3 * torch.randn(rows, 1, generator=g))
    _check_quantized(x.to(dtype).cuda(), 1)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", [(16, 16), (128, 128), (2, 200, 272), (3, 129, 1040)])
def test_quantize_tiles(dtype, shape):
    g = torch.Generator().manual_seed(len(shape))
    _check_quantized((torch.randn(*shape, generator=g) * 0.02).to(dtype).cuda(), 128)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_borders(block_rows):
    # zeros, one value, the largest at 448 s and just above, subnormal results,
    # ties between neighbours, the smallest and the largest fp32 values
    tiny = float(np.finfo(np.float32).smallest_subnormal)
    rows = [[0.0] * 16, [448.0] + [1.0] * 15, [np.nextafter(np.float32(448), np.float32(1e9))] + [1.0] * 15,
            [448.0 * 2.0 ** 20] + [2.0 ** (10 - i) * 1.0625 for i in range(15)],
            [3.4e38] + [1e30] * 15, [tiny] * 16, [1e-37] + [-1e-38] * 15,
            [448.0] + [2.0 ** -6 * (i + 0.5) / 8 for i in range(15)], [-0.875, 0.875] + [0.0] * 14]
    x = np.array(rows, np.float32)
    if block_rows == 128:
        for r in x:
            _check_quantized(_cuda(r[None]), 128)
    else:
        _check_quantized(_cuda(x), 1)


# --------------------------------------------------------------- product --
def _choice(rng, B, E, k, empty=0.0, few=0):
    """Random distinct experts per token; some tokens none; only the first
    `few` experts when given."""
    sel = np.full((B, k), -1, np.int32)
    for t in range(B):
        if rng.random() >= empty:
            n = min(k, few or E)
            sel[t, :n] = rng.permutation(few or E)[:n]
    w = np.where(sel >= 0, rng.random((B, k)) + 0.1, 0.0).astype(np.float32)
    return sel, w


def _lists(sel, w, E):
    L = bc.lists_of(sel, w, E)
    dev = {"n_active": _cuda(np.array([L["n_active"], 0, 0, 0], np.int32)), "active": _cuda(L["active"]),
           "offsets": _cuda(L["offsets"]), "tok": _cuda(L["tok"]), "w": _cuda(L["w"].astype(np.float32))}
    return L, dev


def _weights(rng, E, rows, cols):
    """e4m3 bytes and fp32 scales as a checkpoint holds them, and their 64-bit
    values."""
    b = rng.integers(0, 256, (E, rows, cols)).astype(np.uint8)
    b = np.where((b & 0x7F) == 0x7F, 0x30, b).astype(np.uint8)
    b = np.where(rng.random(b.shape) < 0.7, b & 0xBF, b).astype(np.uint8)  # mostly below 2
    s = (0.02 * (0.5 + rng.random((E, -(-rows // 128), -(-cols // 128))))).astype(np.float32)
    v = np.stack([bc.e4m3_decode(b[e]) * np.repeat(np.repeat(s[e].astype(np.float64), 128, 0)[:rows], 128, 1)[:, :cols]
                  for e in range(E)])
    return _cuda(b), _cuda(s), v


def _gemm_case(B, d, E, k, F, y_dtype, empty=0.0, few=0, seed=0):
    rng = np.random.default_rng([seed, B, d, E, k, F])
    sel, w = _choice(rng, B, E, k, empty, few)
    L, dev = _lists(sel, w, E)
    x = torch.from_numpy(rng.standard_normal((B, d)).astype(np.float32)).cuda()
    q, s = moe.moe_quantize_blocks(x)
    Wq, Ws, Wv = _weights(rng, E, F, d)
    ws = moe.new_gemm_workspace()
    y = torch.full((B * k, F), 7.0, dtype=y_dtype, device="cuda")
    moe.moe_expert_gemm_blocks(q, s, Wq, Ws, dev, k, ws=ws, y=y)
    assert moe.moe_check_error(ws) == 0
    xv = _values(q) * bc.spread(s.cpu().numpy().astype(np.float64), B, d, 1)
    got = y.double().cpu().numpy()
    worst = 0.0
    for _, e, lo, hi in bc.entries(L):
        a = xv[L["tok"][lo:hi]]
        ref = a @ Wv[e].T
        tol = bc.sum_bound(d, np.abs(a) @ np.abs(Wv[e]).T) + bc.HALF_STEP["bf16" if y_dtype == BF16 else "f32"] * np.abs(ref)
        assert np.all(np.abs(got[lo:hi] - ref) <= tol), f"expert {e}: {np.max(np.abs(got[lo:hi] - ref) / tol)} of the bound"
        worst = max(worst, float(np.linalg.norm(got[lo:hi] - ref) / np.linalg.norm(ref)))
    assert np.all(got[L["offsets"][-1]:] == 7.0)  # rows behind the last entry
    return worst


@pytest.mark.parametrize("y_dtype", [F32, BF16])
@pytest.mark.parametrize("B,d,E,k,F", [
    (1, 16, 1, 1, 16), (1, 128, 4, 2, 128), (3, 272, 5, 3, 400), (33, 1040, 8, 4, 272), (129, 256, 3, 2, 256),
    (300, 512, 2, 1, 640), (130, 144, 1, 1, 1040), (5, 4096, 16, 8, 144), (600, 1040, 3, 2, 400),
    (1000, 128, 1, 1, 4096), (257, 272, 2, 2, 16), (32, 272, 1, 1, 400), (31, 128, 2, 2, 128), (34, 256, 1, 1, 128),
    (60, 256, 6, 2, 512), (61, 256, 6, 2, 512)])
def test_gemm(B, d, E, k, F, y_dtype):
    worst = _gemm_case(B, d, E, k, F, y_dtype)
    print(f"relative error {worst:.2e}")


def test_gemm_empty_tokens_and_experts():
    _gemm_case(40, 256, 12, 3, 256, BF16, empty=0.4, few=5)
    _gemm_case(9, 256, 512, 16, 128, BF16, empty=0.2)


def test_gemm_no_entries():
    _gemm_case(4, 128, 4, 2, 128, BF16, empty=1.1)


# ------------------------------------------------------------------- FFN --
def _ffn_setup(B, d, E, k, F, x_dtype, empty=0.0, few=0, seed=1):
    rng = np.random.default_rng([seed, B, d, E, k, F])
    sel, w = _choice(rng, B, E, k, empty, few)
    L, dev = _lists(sel, w, E)
    x = torch.from_numpy(rng.standard_normal((B, d)).astype(np.float32)).to(x_dtype).cuda()
    mats = [_weights(rng, E, F, d), _weights(rng, E, F, d), _weights(rng, E, d, F)]
    args = [t for m in mats for t in m[:2]]
    return L, dev, x, args, [m[2] for m in mats]


def _check_ffn(y, x, L, vals, what=""):
    B = x.shape[0]
    ref, bound = bc.ffn(x.double().cpu().numpy(), vals, L, B)
    tol = bound + bc.HALF_STEP["bf16" if y.dtype == BF16 else "f32"] * np.abs(ref) + 1e-30
    err = np.abs(y.double().cpu().numpy() - ref)
    assert np.all(err <= tol), f"{what}: {np.max(err / tol)} of the bound"
    return float(np.linalg.norm(err) / max(np.linalg.norm(ref), 1e-30))


@pytest.mark.parametrize("x_dtype,y_dtype", [(BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("B,d,E,k,F", [
    (1, 16, 1, 1, 16), (1, 256, 4, 2, 128), (4, 272, 6, 3, 144), (17, 512, 8, 4, 256), (130, 256, 2, 2, 272),
    (40, 1040, 40, 5, 400), (300, 128, 3, 1, 128), (700, 512, 4, 2, 384), (260, 272, 1, 1, 144),
    (32, 256, 1, 1, 384), (33, 256, 1, 1, 384), (100, 256, 20, 4, 256)])
def test_ffn(B, d, E, k, F, x_dtype, y_dtype):
    L, dev, x, args, vals = _ffn_setup(B, d, E, k, F, x_dtype)
    ws = moe.new_blocks_workspace(B, d, E, k, F)
    y = moe.moe_expert_ffn_blocks(x, *args, dev, k, ws=ws, y_dtype=y_dtype)
    assert moe.moe_check_error(ws) == 0
    print(f"relative error {_check_ffn(y, x, L, vals):.2e}")
    # deterministic, also in a used workspace
    y2 = moe.moe_expert_ffn_blocks(x, *args, dev, k, ws=ws, y_dtype=y_dtype)
    assert torch.equal(y, y2)


def test_ffn_empty_tokens():
    L, dev, x, args, vals = _ffn_setup(21, 256, 9, 3, 256, BF16, empty=0.5, few=4)
    y = moe.moe_expert_ffn_blocks(x, *args, dev, 3)
    _check_ffn(y, x, L, vals)
    alone = np.setdiff1d(np.arange(21), L["tok"][:L["offsets"][-1]])
    assert len(alone) and torch.all(y[torch.from_numpy(alone).cuda()] == 0)


@pytest.mark.parametrize("E", [6, 64])  # many entries an expert on average, and few
def test_skewed_batches(E):
    # most tokens on two experts, the rest with a handful each: tiles of every
    # fill
    rng = np.random.default_rng(5)
    B, d, k, F = 500, 256, 2, 256
    sel = np.full((B, k), -1, np.int32)
    sel[:, 0] = np.where(np.arange(B) < 300, 1, 4)
    sel[::7, 1] = 2
    sel[3, 1], sel[480, 1] = 0, 5
    w = np.where(sel >= 0, rng.random((B, k)) + 0.1, 0.0).astype(np.float32)
    L, dev = _lists(sel, w, E)
    x = torch.from_numpy(rng.standard_normal((B, d)).astype(np.float32)).cuda()
    mats = [_weights(rng, E, F, d), _weights(rng, E, F, d), _weights(rng, E, d, F)]
    ws = moe.new_blocks_workspace(B, d, E, k, F)
    y = moe.moe_expert_ffn_blocks(x, *[t for m in mats for t in m[:2]], dev, k, ws=ws)
    assert moe.moe_check_error(ws) == 0
    _check_ffn(y, x, L, [m[2] for m in mats])


def test_ffn_no_entries_is_zero():
    L, dev, x, args, _ = _ffn_setup(5, 128, 4, 2, 128, BF16, empty=1.1)
    y = torch.full((5, 128), 3.0, dtype=BF16, device="cuda")
    moe.moe_expert_ffn_blocks(x, *args, dev, 2, y=y)
    assert torch.all(y == 0)


def test_ffn_nan_in_unlisted_tokens_stays_there():
    L, dev, x, args, vals = _ffn_setup(12, 256, 4, 2, 128, F32, empty=0.5)
    clean = x.clone()
    listed = set(L["tok"][:L["offsets"][-1]].tolist())
    for t in range(12):
        if t not in listed:
            x[t] = float("nan")
    y = moe.moe_expert_ffn_blocks(x, *args, dev, 2)
    _check_ffn(y, clean, L, vals)


def test_ffn_on_a_side_stream_and_captured():
    L, dev, x, args, vals = _ffn_setup(20, 256, 6, 3, 256, BF16)
    ws = moe.new_blocks_workspace(20, 256, 6, 3, 256)
    y = torch.zeros(20, 256, dtype=BF16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        moe.moe_expert_ffn_blocks(x, *args, dev, 3, ws=ws, y=y)
    side.synchronize()
    want = y.clone()
    _check_ffn(want, x, L, vals)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_expert_ffn_blocks(x, *args, dev, 3, ws=ws, y=y)
    for _ in range(3):
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    x.copy_(-x)  # the graph reads what the buffers hold at replay
    g.replay()
    _check_ffn(y, x, L, vals)


@pytest.mark.parametrize("field,value", [("n_active", -1), ("n_active", 99), ("active", 6), ("active", -2),
                                         ("offsets", 10 ** 6), ("offsets", -3), ("tok", 20), ("tok", -1)])
def test_bad_lists_are_reported(field, value):
    L, dev, x, args, vals = _ffn_setup(20, 256, 6, 3, 256, BF16)
    ws = moe.new_blocks_workspace(20, 256, 6, 3, 256)
    keep = dev[field].clone()
    dev[field][1 if field == "offsets" else 0] = value
    moe.moe_expert_ffn_blocks(x, *args, dev, 3, ws=ws)
    assert moe.moe_check_error(ws) == 6
    gws = moe.new_gemm_workspace()
    q, s = moe.moe_quantize_blocks(x)
    moe.moe_expert_gemm_blocks(q, s, args[0], args[1], dev, 3, ws=gws)
    assert moe.moe_check_error(gws) == 6
    dev[field].copy_(keep)
    y = moe.moe_expert_ffn_blocks(x, *args, dev, 3, ws=ws)
    assert moe.moe_check_error(ws) == 0
    _check_ffn(y, x, L, vals)


# ------------------------------------------------- workspaces and waits --
@pytest.mark.parametrize("B,E", [(20, 6), (150, 4)])  # tiles of 16 and of 128 entries
def test_an_expired_wait_is_reported_and_the_device_stays_usable(B, E):
    d, k, F = 512, 3, 256
    L, dev, x, args, vals = _ffn_setup(B, d, E, k, F, BF16)
    ws, gws = moe.new_blocks_workspace(B, d, E, k, F), moe.new_gemm_workspace()
    q, s = moe.moe_quantize_blocks(x)
    torch.cuda.synchronize()
    try:
        moe.moe_set_wait_limit_ns(1)
        moe.moe_expert_ffn_blocks(x, *args, dev, k, ws=ws)
        assert moe.moe_check_error(ws) == 6
        moe.moe_expert_gemm_blocks(q, s, args[0], args[1], dev, k, ws=gws)
        assert moe.moe_check_error(gws) == 6
    finally:
        moe.moe_set_wait_limit_ns(0)
    ws.zero_()
    gws.zero_()
    y = moe.moe_expert_ffn_blocks(x, *args, dev, k, ws=ws)
    assert moe.moe_check_error(ws) == 0
    _check_ffn(y, x, L, vals)


def test_one_workspace_for_calls_of_other_sizes():
    cases = [_ffn_setup(B, d, E, k, F, BF16, seed=B) + (k,) for B, d, E, k, F in
             [(70, 512, 8, 3, 256), (3, 128, 4, 2, 384), (200, 256, 2, 2, 128), (1, 1024, 8, 8, 256)]]
    ws = torch.zeros(max(moe.new_blocks_workspace(c[2].shape[0], c[2].shape[1], c[3][0].shape[0], c[5],
                                                  c[3][0].shape[1]).numel() for c in cases), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        for L, dev, x, args, vals, k in cases:
            y = moe.moe_expert_ffn_blocks(x, *args, dev, k, ws=ws)
            _check_ffn(y, x, L, vals)
    assert moe.moe_check_error(ws) == 0


def test_two_streams_at_once():
    a, b = _ffn_setup(90, 512, 4, 2, 512, BF16, seed=3), _ffn_setup(12, 512, 16, 4, 512, BF16, seed=4)
    k = (2, 4)
    want = [moe.moe_expert_ffn_blocks(c[2], *c[3], c[1], n) for c, n in zip((a, b), k)]
    ws = [moe.new_blocks_workspace(90, 512, 4, 2, 512), moe.new_blocks_workspace(12, 512, 16, 4, 512)]
    ys = [torch.empty_like(w) for w in want]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(30):
        for i, c in enumerate((a, b)):
            moe.moe_expert_ffn_blocks(c[2], *c[3], c[1], k[i], ws=ws[i], y=ys[i], stream=streams[i])
    torch.cuda.synchronize()
    for i, c in enumerate((a, b)):
        assert moe.moe_check_error(ws[i]) == 0
        assert torch.equal(ys[i], want[i])
    _check_ffn(want[0], a[2], a[0], a[4])
    _check_ffn(want[1], b[2], b[0], b[4])


def test_two_captured_graphs_take_turns_in_one_workspace():
    a, b = _ffn_setup(30, 256, 4, 2, 256, BF16, seed=5), _ffn_setup(150, 256, 4, 2, 256, BF16, seed=6)
    ws = moe.new_blocks_workspace(150, 256, 4, 2, 256)
    ys = [torch.zeros(30, 256, dtype=BF16, device="cuda"), torch.zeros(150, 256, dtype=BF16, device="cuda")]
    graphs = []
    for c, y in zip((a, b), ys):
        moe.moe_expert_ffn_blocks(c[2], *c[3], c[1], 2, ws=ws, y=y)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.moe_expert_ffn_blocks(c[2], *c[3], c[1], 2, ws=ws, y=y)
        graphs.append(g)
    for y in ys:
        y.zero_()
    for i in (0, 1, 0, 0, 1):
        graphs[i].replay()
    torch.cuda.synchronize()
    assert moe.moe_check_error(ws) == 0
    _check_ffn(ys[0], a[2], a[0], a[4])
    _check_ffn(ys[1], b[2], b[0], b[4])


# ------------------------------------------------------- long and chained --
def test_quantize_past_two_to_the_31():
    rows, cols = 33000, 65536
    x = torch.zeros(rows, cols, dtype=BF16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    for r in (0, 16384, 32767, 32768, 32999):
        x[r] = torch.randn(cols, device="cuda", generator=g).to(BF16)
    q, s = moe.moe_quantize_blocks(x)
    for r in (0, 1, 16384, 32767, 32768, 32998, 32999):
        rq, rs = bc.quantize(x[r:r + 1].double().cpu().numpy())
        assert np.array_equal(_values(q[r:r + 1]), rq) and np.array_equal(s[r:r + 1].double().cpu().numpy(), rs)


def test_ffn_past_two_to_the_31():
    # B * k * d = 2.2e9 values of dispatched rows and of down products
    B, d, E, k, F = 17000, 16384, 8, 8, 16
    rng = np.random.default_rng(9)
    sel = np.tile(np.arange(8, dtype=np.int32), (B, 1))
    w = (rng.random((B, k)) + 0.1).astype(np.float32)
    tok = np.tile(np.arange(B, dtype=np.int32), E)
    dev = {"n_active": _cuda(np.array([E, 0, 0, 0], np.int32)), "active": _cuda(np.arange(E, dtype=np.int32)),
           "offsets": _cuda((np.arange(E + 1) * B).astype(np.int32)), "tok": _cuda(tok), "w": _cuda(w.T.reshape(-1))}
    x = torch.randn(B, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(BF16)
    mats = [_weights(rng, E, F, d), _weights(rng, E, F, d), _weights(rng, E, d, F)]
    ws = moe.new_blocks_workspace(B, d, E, k, F)
    y = moe.moe_expert_ffn_blocks(x, *[t for m in mats for t in m[:2]], dev, k, ws=ws)
    assert moe.moe_check_error(ws) == 0
    at = np.array([0, 1, 8191, 16383, 16998, 16999])
    L = bc.lists_of(sel[at], w[at], E)
    _check_ffn(y[torch.from_numpy(at).cuda()], x[torch.from_numpy(at).cuda()], L, [m[2] for m in mats])


@pytest.mark.parametrize("B", [1, 37, 200])
def test_router_scored_router_and_both_expert_ffns(B):
    # as a layer uses them: logits, choice and lists, then the experts in 8
    # bits and, from the same lists, in bf16
    d, E, k, F = 512, 32, 4, 256
    rng = np.random.default_rng([11, B])
    x = torch.from_numpy(rng.standard_normal((B, d)).astype(np.float32)).cuda()
    Wg = torch.from_numpy((rng.standard_normal((E, d)) * 0.05).astype(np.float32)).cuda()
    beta = torch.from_numpy((rng.standard_normal(E) * 0.05).astype(np.float32)).cuda()
    logits, _, _, _ = moe.moe_route(x, Wg, None, k)
    sel, w, lists = moe.moe_route_scored(logits, k, moe.MOE_SCORE_SIGMOID, bias=beta, groups=4, top_groups=2,
                                         group_best=2, scale=2.5)
    rsel, rw = bc.route(logits.cpu().numpy(), k, True, beta.cpu().numpy(), 4, 2, 2, True, 2.5)
    assert np.array_equal(sel.cpu().numpy(), rsel)
    L = bc.lists_of(rsel, w.cpu().numpy(), E)
    W = [torch.from_numpy((rng.standard_normal((E, r, c)) * 0.05).astype(np.float32)).cuda()
         for r, c in ((F, d), (F, d), (d, F))]
    quant = [moe.moe_quantize_blocks(m, 128) for m in W]
    vals = [np.stack([v * bc.spread(t, *v.shape, 128) for v, t in zip(_values(q), s.double().cpu().numpy())])
            for q, s in quant]
    ws = moe.new_blocks_workspace(B, d, E, k, F)
    y = moe.moe_expert_ffn_blocks(x, *[t for m in quant for t in m], lists, k, ws=ws)
    assert moe.moe_check_error(ws) == 0
    _check_ffn(y, x, L, vals)
    yb = moe.moe_expert_ffn(x, *[m.to(BF16).view(torch.int16) for m in W], lists, k, moe.new_workspace(B, d, E, k, F))
    # e4m3 keeps three bits: x, the weights and h are each off by 2^-4 of
    # themselves at most, and the errors are independent
    assert float((y - yb).norm() / yb.norm()) < 4 * 2.0 ** -4
