"""The router's losses and their gradient on the GPU against the fp64 oracle.

Bounds.  An exponential is the hardware's base-2 one (off by two steps of 2^-23) of
x log2(e), which log2(e)'s own rounding and the product's move by less than a
step for each |x|, x a logit less the row's largest: less than 2 + 1.173 |x| steps
of 2^-23; so p, a quotient of one and a sum of E of them, by twice that (R below)
and the sum's and the quotient's own log2(32) + 8 + 3 half steps.  Means over
tokens add positive terms in chains of at most 32 tokens, 32 groups of a block,
segments by halves and one quotient: 128 half steps.  logsumexp is off by the sum's
relative error and two half steps of its own magnitude; squares and their sum
twice that and the chain's.  A gradient is a handful of products and sums of the
terms whose magnitudes the oracle adds up, each with p's and logsumexp's error."""
import math

import numpy as np
import pytest
import torch

import oracle.training_oracle as O

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

U = O.U32


def spread(logits):
    """Largest distance of a finite logit from its row's top."""
    top = logits.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        d = np.where(np.isfinite(logits) & np.isfinite(top), top - logits, 0.0)
    return d.max() if d.size else 0.0


def p_error(logits):
    return 2 * (2 + 1.173 * spread(logits)) * 2 * U + 16 * U


def make(T, E, k, S=1, seed=0, masked=False, off=False, scale=2.0):
    rng = np.random.default_rng(seed)
    logits = (scale * rng.standard_normal((T, E)) + rng.standard_normal(E)).astype(np.float32)
    if off and E > k:
        logits[:, E // 2] = -np.inf
    idx = np.argsort(-logits, axis=1, kind="stable")[:, :k].astype(np.int32)
    mask = rng.random(T) > 0.2 if masked else None
    offsets = None
    if S > 1:
        cuts = np.sort(rng.integers(0, T + 1, S - 1))
        offsets = np.concatenate([[T // 50], np.maximum(cuts, T // 50), [T - T // 16]])
        offsets = np.maximum.accumulate(np.minimum(offsets, T - T // 16)).astype(np.int32)
    return logits, idx, mask, offsets


def gpu(v, dtype=None):
    return None if v is None else torch.as_tensor(np.ascontiguousarray(v), device="cuda",
                                                  dtype=dtype)


def forward(logits, idx, S, balance, z, mask=None, offsets=None):
    import moe_expert_mlp_gb300 as m
    T, E = logits.shape
    desc = m.make_router_loss_desc(T, E, idx.shape[1], S, balance, z)
    ws = torch.full((m.moe_router_loss_workspace_size(desc),), 0xCD, dtype=torch.uint8, device="cuda")
    out = dict(counts=torch.full((S, E), -9, dtype=torch.int32, device="cuda"),
               tokens=torch.full((S + 1,), -9, dtype=torch.int32, device="cuda"),
               probs=torch.full((S, E), -9.0, device="cuda"),
               loss=torch.full((3,), -9.0, device="cuda"))
    m.moe_router_loss_fwd(desc, gpu(logits), gpu(idx), gpu(mask), gpu(offsets), out["counts"],
                          out["tokens"], out["probs"], out["loss"], ws)
    return desc, {n: t.cpu().numpy() for n, t in out.items()}, out


def check_forward(logits, idx, S, balance, z, mask, offsets, got):
    l64 = logits.astype(np.float64)
    counts, tokens, probs, loss, zmag = O.router_loss(l64, idx, S, balance, z, mask, offsets)
    assert np.array_equal(got["counts"], counts) and np.array_equal(got["tokens"], tokens)
    rel = p_error(logits) + 128 * U
    assert np.all(np.abs(got["probs"] - probs) <= rel * probs + 1e-37)
    zerr = 2 * zmag * p_error(logits) + (4 + 128) * U * loss[2]
    assert abs(got["loss"][1] - loss[1]) <= (rel + U) * loss[1]
    assert abs(got["loss"][2] - loss[2]) <= zerr
    assert abs(got["loss"][0] - loss[0]) <= (abs(balance) * (rel + U) * loss[1] + abs(z) * zerr +
                                             2 * U * (abs(balance) * loss[1] + abs(z) * loss[2]))


SIZES = [(1, 1, 1), (1, 256, 8), (2, 8, 2), (31, 7, 3), (32, 8, 2), (33, 9, 2), (255, 32, 4),
         (256, 33, 32), (257, 64, 6), (258, 65, 1), (1000, 61, 4), (1001, 128, 8), (777, 129, 5),
         (4099, 130, 2), (3001, 252, 8), (20000, 256, 8), (9000, 4, 1), (70000, 3, 2)]


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("S,masked,off", [(1, False, False), (1, True, True), (4, False, True),
                                          (7, True, False)])
def test_forward(T, E, k, S, masked, off):
    logits, idx, mask, offsets = make(T, E, k, S, T + E, masked, off)
    _, got, _ = forward(logits, idx, S, 0.5, 0.25, mask, offsets)
    check_forward(logits, idx, S, 0.5, 0.25, mask, offsets, got)


def backward(desc, logits, idx, mask, offsets, out, dloss=None, routed=None, offset=0):
    import moe_expert_mlp_gb300 as m
    T, E = logits.shape
    room = torch.full((T * E + 2 * offset,), -9.0, device="cuda")
    dlogits = room[offset:offset + T * E].view(T, E)
    if routed is not None:
        routed = dict(dw=gpu(routed[0]), topk_w=gpu(routed[1]), topk_idx=gpu(routed[2]))
    m.moe_router_loss_bwd(desc, gpu(logits), gpu(mask), gpu(offsets), out["counts"], out["tokens"],
                          dloss, routed, dlogits)
    return dlogits.cpu().numpy().astype(np.float64)


def check_backward(logits, k, S, balance, z, mask, offsets, out, got, dloss, routed):
    ref, mag = O.router_loss_grad(
        logits.astype(np.float64), k, S, out["counts"], out["tokens"], balance, z, mask, offsets,
        dloss, None if routed is None else tuple(np.asarray(v, np.float64) if i < 2 else v
                                                 for i, v in enumerate(routed)))
    # p's error reaches a term through p itself, <f, p> and logsumexp
    bound = (3 * p_error(logits) + (24 + k) * U) * mag
    assert np.all(np.abs(got - ref) <= bound + 1e-37)


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("S,masked,off,join", [(1, False, False, True), (1, True, True, False),
                                               (4, False, True, True), (7, True, False, True)])
def test_backward(T, E, k, S, masked, off, join):
    logits, idx, mask, offsets = make(T, E, k, S, 3 * T + E, masked, off)
    desc, got, out = forward(logits, idx, S, 0.5, 0.25, mask, offsets)
    rng = np.random.default_rng(5)
    routed = None
    if join:
        w = rng.random((T, k)).astype(np.float32)
        routed = ((rng.standard_normal((T, k)) / T).astype(np.float32),
                  (w / w.sum(axis=1, keepdims=True)).astype(np.float32), idx)
    dloss = torch.full((1,), 3.0, device="cuda") if join else None
    d = backward(desc, logits, idx, mask, offsets, out, dloss, routed, offset=E % 4)
    check_backward(logits, k, S, 0.5, 0.25, mask, offsets, got, d, 3.0 if join else 1.0, routed)


def test_gradient_of_the_weights_alone_is_the_routers_backward():
    import moe_expert_mlp_gb300 as m
    T, E, k = 300, 24, 3
    logits, idx, _, _ = make(T, E, k)
    rng = np.random.default_rng(2)
    w, dw = (rng.standard_normal((T, k)).astype(np.float32) for _ in range(2))
    desc, _, out = forward(logits, idx, 1, 0.0, 0.0)
    got = backward(desc, logits, idx, None, None, out, None, (dw, w, idx))
    plain = torch.empty((T, E), device="cuda")
    m.moe_route_bwd(m.make_desc(T, E, k, 64, 32), gpu(dw), gpu(w), gpu(idx), plain)
    ref = plain.cpu().numpy()
    size = np.abs(w) * (np.abs(dw) + np.abs(w * dw).sum(axis=1, keepdims=True))
    assert np.all(np.abs(got - ref) <= 4 * k * U * size.max(axis=1, keepdims=True))
    assert np.array_equal(got == 0, ref == 0)


def test_one_expert_named_twice_is_added_twice_in_order():
    T, E, k = 70, 12, 5
    logits, _, _, _ = make(T, E, k)
    rng = np.random.default_rng(3)
    idx = rng.integers(0, 3, (T, k)).astype(np.int32)
    w, dw = (rng.standard_normal((T, k)).astype(np.float32) for _ in range(2))
    desc, got, out = forward(logits, idx, 1, 0.1, 0.0)
    assert np.array_equal(got["counts"][0], np.bincount(idx.ravel(), minlength=E))
    d = backward(desc, logits, idx, None, None, out, None, (dw, w, idx))
    check_backward(logits, k, 1, 0.1, 0.0, None, None, got, d, 1.0, (dw, w, idx))
    assert np.array_equal(d, backward(desc, logits, idx, None, None, out, None, (dw, w, idx)))


def test_rows_without_logits_and_large_logits():
    T, E, k = 200, 40, 4
    logits, idx, _, _ = make(T, E, k, scale=30.0)
    logits[7] = -np.inf
    logits[8, 1:] = -np.inf
    logits[9] = 3e38 * np.sign(logits[9])
    desc, got, out = forward(logits[:9], idx[:9], 1, 1.0, 1e-3)
    check_forward(logits[:9], idx[:9], 1, 1.0, 1e-3, None, None, got)
    d = backward(desc, logits[:9], idx[:9], None, None, out)
    check_backward(logits[:9], k, 1, 1.0, 1e-3, None, None, got, d, 1.0, None)
    assert not d[7].any() and np.count_nonzero(d[8]) <= 1
    # without the z-loss's squares the largest finite logits are fine too
    _, got, out = forward(logits, idx, 1, 1.0, 0.0)
    assert np.isfinite(got["probs"]).all() and np.isfinite(got["loss"][1])


def test_nan_and_inf_stay_in_their_sequence():
    T, E, k = 90, 16, 2
    logits, idx, _, _ = make(T, E, k)
    offsets = np.array([0, 30, 60, 90], np.int32)
    logits[40, 3] = np.nan
    logits[41, 5] = np.inf
    desc, got, out = forward(logits, idx, 3, 1.0, 1.0, None, offsets)
    assert np.isnan(got["loss"]).all() and np.isnan(got["probs"][1]).any()
    assert np.isfinite(got["probs"][[0, 2]]).all()
    d = backward(desc, logits, idx, None, offsets, out)
    assert np.isnan(d[[40, 41]]).all() and np.isfinite(np.delete(d, [40, 41], axis=0)).all()


@pytest.mark.parametrize("T,S,masked", [(0, 1, False), (0, 3, False), (50, 1, True), (50, 3, True),
                                        (3000, 2, True)])
def test_nothing_counted(T, S, masked):
    E, k = 20, 2
    logits, idx, _, _ = make(T, E, k)
    mask = np.zeros(T, bool) if masked else None
    offsets = np.zeros(S + 1, np.int32) if S > 1 else None
    desc, got, out = forward(logits, idx, S, 1.0, 1.0, mask, offsets)
    assert not any(got[n].any() for n in got)
    assert not backward(desc, logits, idx, mask, offsets, out).any()


def test_one_sequence_a_token_and_many_empty_ones():
    T, E, k = 400, 12, 2
    logits, idx, _, _ = make(T, E, k)
    S = 3 * T
    offsets = np.minimum((np.arange(S + 1) + 1) // 3, T).astype(np.int32)
    desc, got, out = forward(logits, idx, S, 1.0, 0.5, None, offsets)
    check_forward(logits, idx, S, 1.0, 0.5, None, offsets, got)
    d = backward(desc, logits, idx, None, offsets, out)
    check_backward(logits, k, S, 1.0, 0.5, None, offsets, got, d, 1.0, None)


def test_mask_of_bytes_and_results_that_repeat():
    T, E, k = 5000, 48, 4
    logits, idx, mask, _ = make(T, E, k, masked=True)
    _, first, _ = forward(logits, idx, 1, 1.0, 1.0, mask)
    _, again, _ = forward(logits, idx, 1, 1.0, 1.0, mask.astype(np.uint8) * 7)
    for n in first:
        assert np.array_equal(first[n], again[n]), n


def test_device_status():
    import moe_expert_mlp_gb300 as m
    T, E, k = 64, 8, 2
    logits, idx, _, _ = make(T, E, k)
    m.moe_read_device_status()
    idx[5, 1] = E
    idx[6, 0] = -1
    desc, got, out = forward(logits, idx, 1, 1.0, 0.0)
    assert m.moe_read_device_status() == 2                      # MOE_DEV_BAD_EXPERT
    assert got["counts"].sum() == T * k - 2 and got["tokens"][0] == T
    w = np.ones((T, k), np.float32)
    assert np.isfinite(backward(desc, logits, idx, None, None, out, None, (w, w, idx))).all()
    assert m.moe_read_device_status() == 2
    forward(logits, np.abs(idx) % E, 2, 1.0, 0.0, None, np.array([0, 40, 30], np.int32))
    assert m.moe_read_device_status() == 1                      # MOE_DEV_BAD_OFFSETS
    assert m.moe_read_device_status() == 0


@pytest.mark.parametrize("T,E", [(300, 64), (9000, 64), (9000, 61), (40000, 256)])
def test_offsets_that_descend_are_only_reported(T, E):
    """Over many rounds of the rows' ring: neither a wait that runs out nor a trace in
    the next call."""
    import moe_expert_mlp_gb300 as m
    k = 2
    logits, idx, _, _ = make(T, E, k)
    good = np.array([0, T // 3, T // 2, T], np.int32)
    want = forward(logits, idx, 3, 1.0, 0.0, None, good)[1]
    m.moe_read_device_status()
    for bad in ([0, T, T // 2, T], [T // 2, T // 4, T, 7], [0, 200, 50, T - 1], [T, 0, T, 0]):
        desc, _, out = forward(logits, idx, 3, 1.0, 0.0, None, np.array(bad, np.int32))
        assert m.moe_read_device_status() == 1                  # MOE_DEV_BAD_OFFSETS
        backward(desc, logits, idx, None, np.array(bad, np.int32), out, None, None)
        assert m.moe_read_device_status() == 0
    again = forward(logits, idx, 3, 1.0, 0.0, None, good)[1]
    assert all(np.array_equal(want[n], again[n]) for n in want)


def test_graph_and_other_stream():
    """Captured on a stream of its own and replayed on new values."""
    import moe_expert_mlp_gb300 as m
    T, E, k, S = 900, 40, 3, 3
    logits, idx, mask, offsets = make(T, E, k, S, masked=True)
    desc = m.make_router_loss_desc(T, E, k, S, 0.7, 0.1)
    g = dict(logits=gpu(logits), idx=gpu(idx), mask=gpu(mask), offsets=gpu(offsets))
    out = dict(counts=torch.zeros((S, E), dtype=torch.int32, device="cuda"),
               tokens=torch.zeros(S + 1, dtype=torch.int32, device="cuda"),
               probs=torch.zeros((S, E), device="cuda"), loss=torch.zeros(3, device="cuda"))
    dlogits = torch.zeros((T, E), device="cuda")
    ws = torch.empty(m.moe_router_loss_workspace_size(desc), dtype=torch.uint8, device="cuda")

    def step(stream):
        m.moe_router_loss_fwd(desc, g["logits"], g["idx"], g["mask"], g["offsets"], out["counts"],
                              out["tokens"], out["probs"], out["loss"], ws, stream)
        m.moe_router_loss_bwd(desc, g["logits"], g["mask"], g["offsets"], out["counts"],
                              out["tokens"], None, None, dlogits, stream)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    step(stream)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step(torch.cuda.current_stream())
    for seed in (11, 12):
        new, idx, _, _ = make(T, E, k, S, seed)
        g["logits"].copy_(gpu(new))
        g["idx"].copy_(gpu(idx))
        graph.replay()
        torch.cuda.synchronize()
        got = {n: t.cpu().numpy() for n, t in out.items()}
        check_forward(new, idx, S, 0.7, 0.1, mask, offsets, got)
        check_backward(new, k, S, 0.7, 0.1, mask, offsets, got,
                       dlogits.cpu().numpy().astype(np.float64), 1.0, None)
