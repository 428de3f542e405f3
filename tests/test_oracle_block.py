"""The fp64 oracle of the residual block's norms and of gradient clipping,
pinned by closed forms, torch's own layer norm, autograd of an independent
forward, and central differences."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B


def rng(seed=0):
    return np.random.default_rng(seed)


def test_rms_norm_closed_form():
    v = np.array([[3.0, -4.0], [0.0, 0.0], [1e-9, 1e-9]])
    n, mag = B.norm_fwd(v, B.NormSpec("rms", 0.25), np.array([1.0, 2.0]), np.array([0.0, 10.0]))
    assert np.allclose(n[0], [3 / np.sqrt(12.75), -8 / np.sqrt(12.75) + 10])
    assert np.array_equal(n[1], [0.0, 10.0])
    assert np.allclose(mag[0], [3 / np.sqrt(12.75), 8 / np.sqrt(12.75) + 10])
    # weights stored around zero: offset 1 and w = 0 is the plain norm
    n0, _ = B.norm_fwd(v, B.NormSpec("rms", 0.25, 1.0), np.zeros(2))
    n1, _ = B.norm_fwd(v, B.NormSpec("rms", 0.25))
    assert np.array_equal(n0, n1)


def test_layer_norm_is_torchs():
    g = rng(1)
    v, w, b = g.standard_normal((5, 33)) + 3, g.standard_normal(33), g.standard_normal(33)
    ref = torch.nn.functional.layer_norm(torch.from_numpy(v), (33,), torch.from_numpy(w),
                                         torch.from_numpy(b), 1e-5).numpy()
    n, _ = B.norm_fwd(v, B.NormSpec("layer", 1e-5), w, b)
    assert np.allclose(n, ref, rtol=1e-12, atol=1e-12)


def _forward(t, kinds, gate_kind, gate_act, a, b):
    """x', r' as torch sees them (written apart from the oracle)."""
    def norm(v, kind, w, c):
        if kind is None:
            return v
        if kind == "layer":
            return torch.nn.functional.layer_norm(v, v.shape[1:], w + 0.5, c, 1e-5)
        return v * (v.square().mean(1, keepdim=True) + 1e-5).pow(-0.5) * (w + 0.5) + c

    n = norm(t["y"], kinds[1], t["post_w"], t["post_b"])
    if gate_kind is not None:
        g = {"none": lambda q: q, "sigmoid": torch.sigmoid, "tanh": torch.tanh}[gate_act](t["gate"])
        n = n * (g.unsqueeze(1) if gate_kind == "token" else g)
    r = a * t["res"] + b * n
    return r, norm(r, kinds[0], t["pre_w"], t["pre_b"])


@pytest.mark.parametrize("kinds", [("rms", "rms"), ("layer", "rms"), ("rms", "layer"),
                                   ("layer", None)])
@pytest.mark.parametrize("gate", [(None, "none"), ("channel", "sigmoid"), ("token", "tanh"),
                                  ("full", "none")])
def test_gradients_are_autograds_and_differences(kinds, gate):
    gate_kind, act = gate
    T, d, a, b = 4, 7, 0.75, 0.5
    g = rng(3)
    t = {n: torch.from_numpy(g.standard_normal(s)).requires_grad_() for n, s in
         dict(y=(T, d), res=(T, d), post_w=d, post_b=d, pre_w=d, pre_b=d,
              gate={None: 1, "channel": d, "token": T, "full": (T, d)}[gate_kind]).items()}
    dr, dx = g.standard_normal((T, d)), g.standard_normal((T, d))
    r, x = _forward(t, kinds, gate_kind, act, a, b)
    loss = (r * torch.from_numpy(dr)).sum() + (x * torch.from_numpy(dx)).sum()
    names = list(t)
    ref = dict(zip(names, torch.autograd.grad(loss, [t[n] for n in names], allow_unused=True)))
    q = {n: v.detach().numpy() for n, v in t.items()}
    pre, post = B.NormSpec(kinds[0], 1e-5, 0.5), B.NormSpec(kinds[1], 1e-5, 0.5)
    r64, _ = B.post_fwd(q["res"], q["y"], np.abs(q["y"]), post, q["post_w"], q["post_b"],
                        q["gate"], gate_kind, act, a, b)
    x64, _ = B.norm_fwd(r64, pre, q["pre_w"], q["pre_b"])
    assert np.allclose(r64, r.detach().numpy(), rtol=1e-12, atol=1e-12)
    assert np.allclose(x64, x.detach().numpy(), rtol=1e-12, atol=1e-12)
    (D, mag), dpw, dpb = B.join_grads(dr, dx, r64, pre, q["pre_w"], 1.0)
    out = B.post_bwd(D, mag, q["y"], post, q["post_w"], q["post_b"], q["gate"], gate_kind, act, b)
    got = dict(res=a * D, y=out["dy"][0], pre_w=dpw[0], pre_b=dpb[0])
    if kinds[1] is not None:
        got.update(post_w=out["dw"][0], post_b=out["db"][0])
    if gate_kind is not None:
        got["gate"] = out["gate"][0]
    for n, v in got.items():
        assert np.allclose(v, ref[n].numpy(), rtol=1e-10, atol=1e-10), n
    # central differences of the forward along one random direction
    h = 1e-6
    dirs = {n: g.standard_normal(v.shape) for n, v in q.items()}

    def value(sign):
        moved = {n: torch.from_numpy(v + sign * h * dirs[n]) for n, v in q.items()}
        r1, x1 = _forward(moved, kinds, gate_kind, act, a, b)
        return float((r1 * torch.from_numpy(dr)).sum() + (x1 * torch.from_numpy(dx)).sum())

    slope = (value(1) - value(-1)) / (2 * h)
    inner = sum(float((v * dirs[n]).sum()) for n, v in got.items())
    assert abs(slope - inner) <= 1e-7 * (1 + abs(inner))


def test_combine_rows_by_hand():
    Y = np.array([[1.0, 2.0], [10.0, -20.0], [100.0, 200.0]])
    y, mag = B.combine_rows(Y, np.array([[2, 1], [0, 0]]), np.array([[0.5, 2.0], [1.0, 3.0]]))
    assert np.array_equal(y, [[70.0, 60.0], [4.0, 8.0]])
    assert np.array_equal(mag, [[70.0, 140.0], [4.0, 8.0]])


def test_grad_norm_and_factor():
    g = [np.array([3.0, -4.0]), np.zeros((2, 3)), np.zeros(0), np.array([[12.0]])]
    total, each = B.grad_norm(g)
    assert total == pytest.approx(13.0, rel=1e-15) and np.allclose(each, [5.0, 0.0, 0.0, 12.0])
    total, each = B.grad_norm(g, "inf")
    assert total == 12.0 and np.array_equal(each, [4.0, 0.0, 0.0, 12.0])
    total, _ = B.grad_norm([np.array([3e200, -4e200]), np.array([1e-200])])
    assert total == pytest.approx(5e200, rel=1e-15)
    assert B.grad_norm([])[0] == 0.0
    assert B.clip_factor(13.0, 1.0, 0.0) == 1.0 / 13.0
    assert B.clip_factor(0.5, 1.0, 1e-6) == 1.0
    assert np.isnan(B.clip_factor(np.nan, 1.0, 1e-6)) and B.clip_factor(np.inf, 1.0, 1e-6) == 0.0
