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
