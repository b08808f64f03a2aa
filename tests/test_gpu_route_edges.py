"""moe_route_scored where it can go wrong: scores that fp64 cannot tell apart
or cannot hold, weights to the last bit, the switch between one launch and
two, masked and padded batches on both, and logits of bf16 precision."""
import numpy as np
import pytest
import torch

import aware_expert_routing_moe_b200 as moe
import block_cases as bc

pytestmark = pytest.mark.gpu

# The weight is one rounding of an fp64 value: half a step of fp32, and a few
# roundings of fp64 (2^-53 each) before it; below the normal numbers half of
# the smallest step.
W_TOL, W_LOW = 2.0 ** -24 * (1 + 2.0 ** -20), 2.0 ** -150 * (1 + 2.0 ** -20)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    moe.load_library()
    yield
    torch.cuda.synchronize()


def _logits(B, E, seed, sd=1.5):
    return (np.random.default_rng([seed, B, E]).standard_normal((B, E)) * sd).astype(np.float32)


def _check(logits, k, sigmoid, bias=None, groups=1, top_groups=1, best=1, renorm=True, scale=1.0):
    B, E = logits.shape
    sel, w, lists = moe.moe_route_scored(
        torch.from_numpy(logits).cuda(), k, moe.MOE_SCORE_SIGMOID if sigmoid else moe.MOE_SCORE_SOFTMAX,
        bias=None if bias is None else torch.from_numpy(bias).cuda(), groups=groups, top_groups=top_groups,
        group_best=best, renorm=renorm, scale=scale)
    rsel, rw = bc.route(logits, k, sigmoid, bias, groups, top_groups, best, renorm, float(np.float32(scale)))
    sel, w = sel.cpu().numpy(), w.cpu().numpy().astype(np.float64)
    assert np.array_equal(sel, rsel)
    assert np.all(np.abs(w - rw) <= W_TOL * rw + W_LOW), float(np.max(np.abs(w - rw) / np.maximum(rw, 1e-300)))
    ref = bc.lists_of(sel, w, E)
    assert int(lists["n_active"][0]) == ref["n_active"]
    for n in ("active", "offsets", "tok"):
        assert np.array_equal(lists[n].cpu().numpy(), ref[n]), n
    assert np.array_equal(lists["w"].cpu().numpy().astype(np.float64), ref["w"])
    return sel, w


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm,scale", [(True, 1.0), (True, 2.5), (False, 1.0), (False, 0.3)])
def test_weights_are_rounded_once(sigmoid, renorm, scale):
    _check(_logits(150, 96, 1), 8, sigmoid, renorm=renorm, scale=scale)
    _check(_logits(40, 256, 2, 6.0), 16, sigmoid, np.full(256, 0.1, np.float32), renorm=renorm, scale=scale)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("groups,top", [(1, 1), (4, 2)])
def test_scores_that_fp64_cannot_tell_apart_go_to_the_lower_index(sigmoid, groups, top):
    # exp(1e-20) and exp(0) are the same fp64 number: with a bias of zeros and
    # without one the choice is the lower index
    l = np.full((6, 64), -1.0, np.float32)
    l[0, 0], l[0, 5] = 0.0, 1e-20
    l[1, 40], l[1, 3] = 1e-20, -1e-20
    l[2] = np.linspace(1e-12, 64e-12, 64) * 1e-9
    l[3, 17], l[3, 16] = 1e-30, 0.0
    l[4, 9:13] = [2e-19, 1e-38, 1e-45, 3e-19]
    l[5] = 0.5
    zero = np.zeros(64, np.float32)
    for k in (1, 4):
        a, _ = _check(l, k, sigmoid, None, groups, top)
        b, _ = _check(l, k, sigmoid, zero, groups, top)
        assert np.array_equal(a, b)
    assert a[0, 0] == 0 and a[3, 0] == 16


def test_small_logits_that_fp64_does_tell_apart():
    # steps of 2^-46: scores 1.4e-14 apart, some sixty fp64 steps
    l = np.full((2, 32), -1.0, np.float32)
    l[0, 3:9] = np.arange(6, dtype=np.float32) * np.float32(2.0 ** -46)
    l[1, 3:9] = -np.arange(6, dtype=np.float32) * np.float32(2.0 ** -46)
    for sigmoid in (False, True):
        _check(l, 4, sigmoid)
        _check(l, 4, sigmoid, np.zeros(32, np.float32))


def test_scores_below_fp64_count_as_zero():
    # the bias steers to experts whose softmax scores are below the smallest
    # fp64 number: their weights are zero, as with sigmoid scores
    l = np.array([[0.0, -800.0, -900.0, np.finfo(np.float32).min] + [-1000.0] * 12], np.float32)
    bias = np.array([-2.0, 1.0, 0.5, 0.25] + [0.0] * 12, np.float32)
    for renorm in (True, False):
        sel, w = _check(l, 3, False, bias, renorm=renorm)
        assert sel.tolist() == [[1, 2, 3]] and np.all(w == 0)
    sel, w = _check(np.where(l == 0, -2000, l).astype(np.float32), 3, True, bias)
    assert sel.tolist() == [[1, 2, 3]] and np.all(w == 0)
    # one of the chosen holds all of the weight
    _, w = _check(l, 3, False, np.array([0.0, 1.5, 0.5] + [-1.0] * 13, np.float32), scale=2.5)
    assert w.tolist() == [[0.0, 2.5, 0.0]]


@pytest.mark.parametrize("E,k", [(1, 1), (33, 4), (160, 6), (512, 16)])
@pytest.mark.parametrize("B", [16, 17, 512, 513, 1100])
@pytest.mark.parametrize("masked", [False, True])
def test_one_launch_and_two(B, E, k, masked):
    l = _logits(B, E, 3)
    if masked:
        rng = np.random.default_rng([4, B, E])
        l[rng.random(l.shape) < 0.3] = -np.inf
        l[rng.random(B) < 0.2] = -np.inf
        l[0], l[-1] = np.nan, -np.inf
    _check(l, k, bool(B & 1) != masked)


@pytest.mark.parametrize("B", [3, 513, 2000])
def test_all_tokens_masked(B):
    sel, _ = _check(np.full((B, 40), -np.inf, np.float32), 5, True)
    assert np.all(sel == -1)


@pytest.mark.parametrize("B", [60, 700])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_logits_of_bf16_precision(B, sigmoid):
    l = torch.from_numpy(_logits(B, 256, 5)).bfloat16().float().numpy()
    _check(l, 8, sigmoid)
    _check(l, 8, sigmoid, None, 8, 3, 1)
    _check(l, 8, sigmoid, (np.random.default_rng(6).standard_normal(256) * 0.05).astype(np.float32), 8, 4, 2)


def test_two_launches_captured_and_replayed():
    T, E, k = 1500, 64, 6
    x = torch.from_numpy(_logits(T, E, 7)).cuda()
    out = (torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda"))
    lists, ws = moe.alloc_lists(T, E, k), moe.new_route_workspace(T, E, k)
    call = lambda: moe.moe_route_scored(x, k, out=out, lists=lists, ws=ws)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for seed in (8, 9):
        l = _logits(T, E, seed)
        x.copy_(torch.from_numpy(l))
        g.replay()
        torch.cuda.synchronize()
        rsel, _ = bc.route(l, k, False)
        assert np.array_equal(out[0].cpu().numpy(), rsel)
        ref = bc.lists_of(rsel, out[1].cpu().numpy(), E)
        for n in ("active", "offsets", "tok"):
            assert np.array_equal(lists[n].cpu().numpy(), ref[n]), n


def test_the_largest_batch():
    # 65536 tokens, 512 experts, 16 of them, some tokens masked: the choice is
    # the order of the logits (distinct, no bias), lists by a stable sort
    B, E, k = 65536, 512, 16
    g = torch.Generator(device="cuda").manual_seed(0)
    l = torch.rand(B, E, device="cuda", generator=g).argsort(1).float() * 0.01
    l[::97] = -float("inf")
    sel, w, lists = moe.moe_route_scored(l, k, moe.MOE_SCORE_SIGMOID, scale=2.0)
    val, idx = l.sort(1, descending=True)
    want = torch.where(val[:, :k] > -float("inf"), idx[:, :k], torch.full_like(idx[:, :k], -1))
    assert torch.equal(sel.long(), want)
    s = torch.sigmoid(val[:, :k].double())
    rw = torch.nan_to_num(s / s.sum(1, keepdim=True) * 2.0)
    assert torch.all((w.double() - rw).abs() <= W_TOL * rw)
    flat = torch.where(want < 0, E, want).reshape(-1)
    order = flat.argsort(stable=True)
    n = int((flat < E).sum())
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    assert int(lists["n_active"][0]) == E and torch.all(counts > 0)
    assert torch.equal(lists["active"].long(), torch.arange(E, device="cuda"))
    assert torch.equal(lists["offsets"][1:].long(), counts.cumsum(0)) and int(lists["offsets"][0]) == 0
    assert torch.equal(lists["tok"][:n].long(), order[:n] // k) and torch.all(lists["tok"][n:] == -1)
    assert torch.equal(lists["w"][:n], w.reshape(-1)[order[:n]]) and torch.all(lists["w"][n:] == 0)


@pytest.mark.parametrize("B", [100, 700])
def test_two_streams_at_once(B):
    ls = [torch.from_numpy(_logits(B, E, 20)).cuda() for E in (64, 256)]
    want = [moe.moe_route_scored(l, 8) for l in ls]
    state = [((torch.empty_like(s), torch.empty_like(w)), moe.alloc_lists(B, l.shape[1], 8),
              moe.new_route_workspace(B, l.shape[1], 8)) for l, (s, w, _) in zip(ls, want)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(30):
        for l, (out, lists, ws), st in zip(ls, state, streams):
            moe.moe_route_scored(l, 8, out=out, lists=lists, ws=ws, stream=st)
    torch.cuda.synchronize()
    for (out, lists, ws), (s, w, ref) in zip(state, want):
        assert torch.equal(out[0], s) and torch.equal(out[1], w)
        for n in ("active", "offsets", "tok", "w"):
            assert torch.equal(lists[n], ref[n]), n
