"""Router's losses at the edges of what they take: rows of logits far from zero,
squares whose sum is out of range.

Bounds: those of test_gpu_router_loss.py."""
import numpy as np
import pytest
import torch

from tests.test_gpu_router_loss import backward, check_backward, check_forward, forward, make

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def far_rows(T, E, k, at):
    """A batch of which two rows in three lie around `at`: some steps of fp32 below it
    where those are no more than 64, all alike where they are wider, some of them
    off."""
    logits, idx, _, _ = make(T, E, k, seed=T + E)
    at = np.float32(at)
    step = 2.0 ** (np.floor(np.log2(abs(np.float64(at)))) - 23)
    rng = np.random.default_rng(7)
    far = at - (step if step <= 64 else 0) * rng.integers(0, 4, (T, E))
    far[:, E // 2] = -np.inf
    rows = np.arange(T) % 3 != 0
    logits[rows] = far[rows].astype(np.float32)
    return logits, idx


@pytest.mark.parametrize("at", [2.0 ** 20, 3e7, -3e7, 1e8, -1e9, 1e10, -1e10, 3e15, -1e18])
@pytest.mark.parametrize("T,E,k", [(200, 64, 4), (200, 61, 4), (3000, 64, 4), (900, 256, 8)])
def test_rows_far_from_zero(T, E, k, at):
    logits, idx = far_rows(T, E, k, at)
    desc, got, out = forward(logits, idx, 1, 1.0, 1e-3)
    check_forward(logits, idx, 1, 1.0, 1e-3, None, None, got)
    d = backward(desc, logits, idx, None, None, out)
    check_backward(logits, k, 1, 1.0, 1e-3, None, None, got, d, 1.0, None)


@pytest.mark.parametrize("at", [1e30, -1e30, 9e37, -9.9e37, 3.4028235e38, -3.4028235e38])
@pytest.mark.parametrize("T,E,k", [(200, 64, 4), (200, 61, 4), (3000, 64, 4)])
def test_rows_whose_squares_leave_the_range(T, E, k, at):
    """Rows masked with a large negative number among them: the mean probabilities, the
    balance and its gradient."""
    logits, idx = far_rows(T, E, k, at)
    desc, got, out = forward(logits, idx, 1, 1.0, 0.0)
    near = logits.copy()
    rows = np.arange(T) % 3 != 0
    near[rows] = np.where(np.isneginf(near[rows]), -np.inf, 0.0)     # the same p
    want = forward(near, idx, 1, 1.0, 0.0)[1]
    for n in ("counts", "tokens", "probs"):
        assert np.array_equal(got[n], want[n]), n
    assert got["loss"][1] == want["loss"][1]
    d = backward(desc, logits, idx, None, None, out)
    check_backward(logits, k, 1, 1.0, 0.0, None, None, got, d, 1.0, None)


@pytest.mark.parametrize("T", [400, 5000, 200000])
def test_mean_of_squares_whose_sum_leaves_the_range(T):
    logits, idx, _, _ = make(T, 8, 2)
    logits[:] = np.where(np.arange(8) == 3, 1.5e19, -np.inf)[None].astype(np.float32)
    for S, offsets in ((1, None), (3, np.array([0, T // 3, T // 2, T], np.int32))):
        _, got, _ = forward(logits, idx, S, 0.5, 0.25, None, offsets)
        check_forward(logits, idx, S, 0.5, 0.25, None, offsets, got)
