"""The fp64 oracle of the router's losses and of orthogonalised updates, against
differences and closed forms; and what fp16 operands cost an update."""
import numpy as np
import pytest

import oracle.training_oracle as O


def routing(T, E, k, seed=0):
    rng = np.random.default_rng(seed)
    logits = rng.standard_normal((T, E))
    return logits, np.argsort(-logits, axis=1, kind="stable")[:, :k]


def test_even_routing_has_balance_one():
    T, E = 24, 6
    logits = np.zeros((T, E))
    idx = (np.arange(T)[:, None] + np.arange(2)) % E
    counts, tokens, probs, loss, _ = O.router_loss(logits, idx, 1, 1.0, 0.5)
    assert np.all(counts == T * 2 // E) and list(tokens) == [T, T]
    assert np.allclose(probs, 1 / E) and np.isclose(loss[1], 1.0)
    assert np.isclose(loss[2], np.log(E) ** 2) and np.isclose(loss[0], 1 + 0.5 * np.log(E) ** 2)


def test_one_expert_for_all_has_balance_of_the_experts():
    logits = np.full((5, 4), -80.0)
    logits[:, 2] = 0.0
    _, _, _, loss, _ = O.router_loss(logits, np.full((5, 1), 2), 1, 1.0, 0.0)
    assert np.isclose(loss[1], 4.0)


@pytest.mark.parametrize("S,masked", [(1, False), (3, True)])
def test_gradient_against_differences(S, masked):
    T, E, k = 9, 5, 2
    logits, idx = routing(T, E, k)
    mask = np.arange(T) % 4 != 1 if masked else None
    offsets = None if S == 1 else [1, 4, 4, 8]
    counts, tokens, _, _, _ = O.router_loss(logits, idx, S, 0.3, 0.2, mask, offsets)
    grad, mag = O.router_loss_grad(logits, k, S, counts, tokens, 0.3, 0.2, mask, offsets, dloss=1.7)
    assert np.all(np.abs(grad) <= mag * (1 + 1e-12))

    def loss(x):
        return O.router_loss(x, idx, S, 0.3, 0.2, mask, offsets)[3][0]

    h = 1e-5
    for t in range(T):
        for e in range(E):
            d = np.zeros_like(logits)
            d[t, e] = h
            # (the counts do not change with the logits here: idx is held)
            assert abs(1.7 * (loss(logits + d) - loss(logits - d)) / (2 * h) - grad[t, e]) < 1e-8


def test_a_row_that_is_masked_out_and_an_expert_switched_off():
    logits, idx = routing(6, 4, 1)
    logits[3] = -np.inf
    logits[:, 1] = -np.inf
    counts, tokens, probs, loss, _ = O.router_loss(logits, idx, 1, 1.0, 1.0)
    assert np.isfinite(loss).all() and probs[0, 1] == 0 and np.isclose(probs.sum(), 5 / 6)
    grad, _ = O.router_loss_grad(logits, 1, 1, counts, tokens, 1.0, 1.0)
    assert np.all(grad[3] == 0) and np.all(grad[:, 1] == 0)


@pytest.mark.parametrize("shape", [(4, 4), (3, 7), (9, 2)])
def test_update_acts_on_the_singular_values(shape):
    rng = np.random.default_rng(1)
    g = rng.standard_normal(shape)
    u, s, vt = np.linalg.svd(g, full_matrices=False)
    s = s / (np.linalg.norm(g) + 1e-7)
    a, b, c = O.DEFAULT
    for _ in range(5):
        s = a * s + b * s ** 3 + c * s ** 5
    assert np.allclose(O.orthogonalize(g, scale=0.5), 0.5 * (u * s) @ vt, atol=1e-12)
    assert np.all((s > 0.6) & (s < 1.25))
    assert not O.orthogonalize(np.zeros(shape)).any()


def spectra(rng, shape):
    r, c = shape
    return {"full": rng.standard_normal(shape),
            "rank 3": rng.standard_normal((r, 3)) @ rng.standard_normal((3, c)),
            "falling": rng.standard_normal(shape) * np.arange(1, c + 1) ** -1.0,
            "few large rows": rng.standard_normal(shape) * np.exp(2 * rng.standard_normal((r, 1)))}


@pytest.mark.parametrize("shape,steps,bound", [
    ((64, 64), 5, 5e-3), ((64, 300), 5, 5e-3), ((200, 96), 5, 5e-3), ((128, 128), 8, 1e-2),
    ((16, 16), 8, 1e-2), ((3, 40), 8, 2e-2)])
def test_what_fp16_operands_cost(shape, steps, bound):
    """The documented error of an update, bf16's own rounding (2^-8 at most)
    apart: sqrt(bound^2 - (2^-8)^2).

    The smallest sides may take 2e-2: with one singular value nothing averages
    out.  Near s = 1 a step's roundings are then off by up to 2^-11 (|B| for X's
    operand, |B| for B's, 3 |b + 2 c s^2| for A's) = 2^-11 (2.8 + 2.8 + 3 * 0.8)
    = 4e-3, and the map passes an error on with up to 1.6 there, so that the last
    four steps come to 4e-3 (1 + 1.6 + 2.6 + 4.1) = 3.7e-2 at the very worst; half
    of that is allowed."""
    for seed in range(3):
        rng = np.random.default_rng(seed)
        for name, g in spectra(rng, shape).items():
            ref = O.orthogonalize(g, steps)
            off = np.linalg.norm(O.orthogonalize_rounded(g, steps) - ref) / np.linalg.norm(ref)
            assert off < np.sqrt(bound ** 2 - 2.0 ** -16), (name, off)


@pytest.mark.parametrize("shape", [(64, 160), (300, 130), (200, 450)])
def test_first_two_steps_as_one_cost_no_more(shape):
    """Two steps by polynomials of A are the same update, and stay within what an
    update of five steps may be off by."""
    for seed in range(3):
        rng = np.random.default_rng(seed)
        for name, g in spectra(rng, shape).items():
            ref = O.orthogonalize(g, 5)
            off = np.linalg.norm(O.orthogonalize_rounded(g, 5, joined=True) - ref) / np.linalg.norm(ref)
            assert off < np.sqrt(5e-3 ** 2 - 2.0 ** -16), (name, off)
