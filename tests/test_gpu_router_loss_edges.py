"""Router's losses at the edges of what they take: rows of logits far from zero,
squares whose sum is out of range, losses without a coefficient, arrays off 16-byte
boundaries, chunks of the most tokens, calls from two host threads at once.

Bounds: those of test_gpu_router_loss.py."""
import threading

import numpy as np
import pytest
import torch

from tests.test_gpu_router_loss import backward, check_backward, check_forward, forward, gpu, make

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


def test_two_host_threads_with_layers_of_different_experts():
    """Calls of 132 and of 256 experts run in one kernel; each thread has its own
    stream, workspace and results."""
    import moe_expert_mlp_gb300 as m
    calls = []
    for T, E, k in ((600, 132, 4), (500, 256, 8)):
        logits, idx, _, _ = make(T, E, k, seed=E)
        desc = m.make_router_loss_desc(T, E, k, 1, 1.0, 1e-3)
        t = dict(logits=torch.from_numpy(logits).cuda(), idx=torch.from_numpy(idx).cuda(),
                 counts=torch.zeros((1, E), dtype=torch.int32, device="cuda"),
                 tokens=torch.zeros(2, dtype=torch.int32, device="cuda"),
                 probs=torch.zeros((1, E), device="cuda"), loss=torch.zeros(3, device="cuda"),
                 dlogits=torch.zeros((T, E), device="cuda"),
                 ws=torch.empty(m.moe_router_loss_workspace_size(desc), dtype=torch.uint8,
                                device="cuda"))
        calls.append((desc, t, torch.cuda.Stream()))

    def step(desc, t, stream):
        m.moe_router_loss_fwd(desc, t["logits"], t["idx"], None, None, t["counts"], t["tokens"],
                              t["probs"], t["loss"], t["ws"], stream)
        m.moe_router_loss_bwd(desc, t["logits"], None, None, t["counts"], t["tokens"], None, None,
                              t["dlogits"], stream)

    results = ("counts", "tokens", "probs", "loss", "dlogits")
    torch.cuda.synchronize()
    want = []
    for desc, t, stream in calls:
        step(desc, t, stream)
        torch.cuda.synchronize()
        want.append({n: t[n].clone() for n in results})
    failures = []

    def work(call):
        try:
            for _ in range(4000):
                step(*call)
        except Exception as e:          # reported by the test's own thread
            failures.append(e)

    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert not failures
    for (_, t, _), w in zip(calls, want):
        assert all(torch.equal(t[n], w[n]) for n in results)


@pytest.mark.parametrize("T", [60, 700])
def test_a_loss_without_a_coefficient_is_left_out(T):
    """A row masked with the most negative finite number: its square leaves fp32's range,
    which is no part of a loss that does not ask for it."""
    E, k = 40, 4
    logits, idx, _, _ = make(T, E, k)
    logits[9] = np.finfo(np.float32).min
    _, got, _ = forward(logits, idx, 1, 0.5, 0.0)
    assert np.isposinf(got["loss"][2]) and np.isfinite(got["loss"][1])
    assert got["loss"][0] == np.float32(0.5) * got["loss"][1]
    _, got, _ = forward(logits, idx, 1, 0.0, 0.0)
    assert got["loss"][0] == 0
    _, got, _ = forward(logits, idx, 1, 0.0, 1e-3)
    assert np.isposinf(got["loss"][0])
    logits[9, 3] = np.nan
    for coefficients in ((0.5, 0.0), (0.0, 1e-3), (0.5, 1e-3)):
        assert np.isnan(forward(logits, idx, 1, *coefficients)[1]["loss"]).all()


def apart(v, by):
    """v on the GPU, `by` elements past a 16-byte boundary."""
    v = np.ascontiguousarray(v)
    t = torch.from_numpy(v)
    room = torch.zeros(v.size + 4, dtype=t.dtype, device="cuda")
    view = room[by:by + v.size].view(v.shape)
    view.copy_(t)
    return view


@pytest.mark.parametrize("T,E,k", [(40, 32, 4), (300, 64, 6), (300, 128, 4), (1100, 32, 2),
                                   (1100, 64, 6), (1100, 128, 8), (1100, 256, 8)])
@pytest.mark.parametrize("which,by", [("logits", 1), ("logits", 2), ("dlogits", 3), ("counts", 1),
                                      ("all", 1)])
def test_arrays_that_no_vector_load_reaches(T, E, k, which, by):
    """Rows of whole 16 bytes in arrays that do not start on such a boundary."""
    import moe_expert_mlp_gb300 as m
    S = 3
    logits, idx, mask, offsets = make(T, E, k, S, T + E, masked=True)
    rng = np.random.default_rng(4)
    w = rng.random((T, k)).astype(np.float32)
    dw = (rng.standard_normal((T, k)) / T).astype(np.float32)
    at = {n: by if which in (n, "all") else 0 for n in ("logits", "dlogits", "counts")}
    x = apart(logits, at["logits"])
    desc = m.make_router_loss_desc(T, E, k, S, 0.5, 0.25)
    ws = torch.empty(m.moe_router_loss_workspace_size(desc), dtype=torch.uint8, device="cuda")
    out = dict(counts=apart(np.full((S, E), -9, np.int32), at["counts"]),
               tokens=torch.full((S + 1,), -9, dtype=torch.int32, device="cuda"),
               probs=torch.full((S, E), -9.0, device="cuda"), loss=torch.full((3,), -9.0, device="cuda"))
    dlogits = apart(np.full((T, E), -9, np.float32), at["dlogits"])
    on = dict(idx=gpu(idx), mask=gpu(mask), offsets=gpu(offsets), w=gpu(w), dw=gpu(dw))
    m.moe_router_loss_fwd(desc, x, on["idx"], on["mask"], on["offsets"], out["counts"],
                          out["tokens"], out["probs"], out["loss"], ws)
    m.moe_router_loss_bwd(desc, x, on["mask"], on["offsets"], out["counts"], out["tokens"], None,
                          dict(dw=on["dw"], topk_w=on["w"], topk_idx=on["idx"]), dlogits)
    got = {n: t.cpu().numpy() for n, t in out.items()}
    check_forward(logits, idx, S, 0.5, 0.25, mask, offsets, got)
    check_backward(logits, k, S, 0.5, 0.25, mask, offsets, got,
                   dlogits.cpu().numpy().astype(np.float64), 1.0, (dw, w, idx))
    assert m.moe_read_device_status() == 0


@pytest.mark.parametrize("T,E,k", [(640_001, 8, 2), (320_003, 68, 4)])
def test_chunks_of_the_most_tokens(T, E, k):
    """More tokens than blocks of 1024 hold in one wave."""
    logits, idx, mask, offsets = make(T, E, k, 3, 9, masked=True)
    desc, got, out = forward(logits, idx, 3, 0.5, 0.25, mask, offsets)
    check_forward(logits, idx, 3, 0.5, 0.25, mask, offsets, got)
    d = backward(desc, logits, idx, mask, offsets, out)
    check_backward(logits, k, 3, 0.5, 0.25, mask, offsets, got, d, 1.0, None)
