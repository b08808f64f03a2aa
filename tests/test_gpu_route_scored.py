"""GPU parity of moe_route_scored against a 64-bit restatement: the choice
and the lists exactly, the weights to fp32 rounding."""
import numpy as np
import pytest
import torch

import aware_expert_routing_moe_b200 as moe
import block_cases as bc

pytestmark = pytest.mark.gpu

# fp32 weights: the score, the sum of up to 16 scores, the division and the
# scale each round: at most 2 units of exp and 20 half steps
W_TOL = 24 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    moe.load_library()
    yield
    torch.cuda.synchronize()


def _check(logits, k, sigmoid, bias=None, groups=1, top_groups=1, best=1, renorm=True, scale=1.0):
    B, E = logits.shape
    sel, w, lists = moe.moe_route_scored(
        torch.from_numpy(logits).cuda(), k, moe.MOE_SCORE_SIGMOID if sigmoid else moe.MOE_SCORE_SOFTMAX,
        bias=None if bias is None else torch.from_numpy(bias).cuda(), groups=groups, top_groups=top_groups,
        group_best=best, renorm=renorm, scale=scale)
    rsel, rw = bc.route(logits, k, sigmoid, bias, groups, top_groups, best, renorm, float(np.float32(scale)))
    sel, w = sel.cpu().numpy(), w.cpu().numpy().astype(np.float64)
    assert np.array_equal(sel, rsel)
    assert np.all(np.abs(w - rw) <= W_TOL * rw + 1e-37)
    ref = bc.lists_of(sel, w, E)
    assert int(lists["n_active"][0]) == ref["n_active"]
    for n in ("active", "offsets", "tok"):
        assert np.array_equal(lists[n].cpu().numpy(), ref[n]), n
    assert np.array_equal(lists["w"].cpu().numpy().astype(np.float64), ref["w"])
    return sel


def _logits(B, E, seed, sd=1.5):
    return (np.random.default_rng([seed, B, E]).standard_normal((B, E)) * sd).astype(np.float32)


def _bias(E, seed=3, sd=0.05):
    return (np.random.default_rng([seed, E]).standard_normal(E) * sd).astype(np.float32)


@pytest.mark.parametrize("B", [1, 2, 63, 64, 65, 200])
@pytest.mark.parametrize("E,k", [(1, 1), (8, 8), (16, 3), (33, 4), (128, 8), (160, 6), (256, 8), (512, 16)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_plain(B, E, k, sigmoid):
    _check(_logits(B, E, 0), k, sigmoid)


@pytest.mark.parametrize("B", [1, 37, 300])
@pytest.mark.parametrize("E,k,groups,top", [(16, 2, 4, 2), (60, 6, 4, 2), (128, 8, 16, 5), (256, 8, 8, 4),
                                            (512, 16, 32, 7), (32, 4, 32, 4)])
@pytest.mark.parametrize("best", [1, 2])
def test_groups_and_bias(B, E, k, groups, top, best):
    for sigmoid in (False, True):
        _check(_logits(B, E, 1), k, sigmoid, _bias(E), groups, top, best, scale=2.5)
        _check(_logits(B, E, 2), k, sigmoid, None, groups, top, best, renorm=False)


@pytest.mark.parametrize("B", [9000, 20000])
def test_many_tokens(B):
    _check(_logits(B, 64, 4), 4, True, _bias(64), 8, 3, 2)


@pytest.mark.parametrize("groups,top", [(1, 1), (8, 2)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_masked_logits(groups, top, sigmoid):
    l = _logits(70, 64, 5)
    rng = np.random.default_rng(6)
    l[rng.random(l.shape) < 0.5] = -np.inf
    l[3] = -np.inf                       # nothing left
    l[4] = np.nan
    l[5] = -np.inf
    l[5, 17] = -30.0                     # one expert left
    l[6] = np.finfo(np.float32).min      # a mask of the type's lowest value leaves a choice
    l[7, 5] = np.inf
    l[8, 40:] = -np.inf
    l[9, ::2] = np.nan
    sel = _check(l, 8, sigmoid, _bias(64), groups, top, 2)
    assert np.all(sel[3] == -1) and np.all(sel[4] == -1) and sel[5, 0] == 17 and np.all(sel[5, 1:] == -1)


def test_all_tokens_masked():
    l = np.full((5, 32), -np.inf, np.float32)
    _check(l, 4, False)
    _check(l, 4, True, groups=4, top_groups=2)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_equal_values_go_to_the_lower_index(sigmoid):
    l = np.zeros((40, 96), np.float32)
    l[1:] = np.round(_logits(39, 96, 7) * 2) / 2
    l[2] = -l[2] * 0.0                   # zeros of both signs
    _check(l, 8, sigmoid)
    _check(l, 8, sigmoid, np.zeros(96, np.float32), 8, 3, 2)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_near_ties_are_decided_exactly(sigmoid):
    # logits one fp32 step apart in shuffled order: the scores, and the values
    # with a bias, differ by far less than an fp32 step
    rng = np.random.default_rng(8)
    B, E = 50, 128
    l = np.empty((B, E), np.float32)
    for t in range(B):
        v = np.full(E, np.float32(rng.uniform(-2, 2)), np.float32)
        for e in range(1, E):
            v[e] = np.nextafter(v[e - 1], np.float32(10))
        l[t] = rng.permutation(v)
    _check(l, 8, sigmoid)
    _check(l, 8, sigmoid, np.full(E, 0.7, np.float32))
    _check(l, 8, sigmoid, np.full(E, 0.7, np.float32), 8, 3, 2)
    # a bias that makes up for the score to within fp32 rounding
    x = _logits(1, E, 9)[0]
    s = 1 / (1 + np.exp(-x.astype(np.float64)))
    if not sigmoid:
        s = np.exp(x.astype(np.float64)) / np.exp(x.astype(np.float64)).sum()
    _check(np.repeat(x[None], 4, 0), 8, sigmoid, (1.0 - s).astype(np.float32))


def test_extreme_logits():
    l = np.zeros((4, 32), np.float32)
    l[0] = np.linspace(-100, -80, 32)    # sigmoid scores near the fp32 underflow
    l[1] = np.linspace(-300, 300, 32)
    l[2] = np.linspace(15, 16, 32)       # sigmoid near 1
    _check(l, 4, True)
    _check(l, 4, False)
    _check(l, 4, True, renorm=False)


def test_captured_and_replayed_on_new_logits():
    T, E, k = 100, 128, 8
    x = torch.from_numpy(_logits(T, E, 10)).cuda()
    out = (torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda"))
    lists, ws = moe.alloc_lists(T, E, k), moe.new_route_workspace(T, E, k)
    call = lambda: moe.moe_route_scored(x, k, moe.MOE_SCORE_SIGMOID, out=out, lists=lists, ws=ws)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    l2 = _logits(T, E, 11)
    x.copy_(torch.from_numpy(l2))
    g.replay()
    torch.cuda.synchronize()
    rsel, _ = bc.route(l2, k, True)
    assert np.array_equal(out[0].cpu().numpy(), rsel)
