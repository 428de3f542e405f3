"""Edges of the residual block's norms on the GPU."""
import pytest
import torch

from tests.test_gpu_block_norm import Case

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.mark.parametrize("gate", [None, "channel", "token", "full"])
def test_no_tokens_with_every_gate(gate):
    """T = 0: the parameters' gradients are zero whatever the gate."""
    c = Case(T=0, d=96, gate=gate, bias=True)
    none = torch.empty(0, 96, dtype=c.at, device="cuda")
    c.m.moe_block_post_norm_fwd(c.desc, none, none, c.p, none, none)
    grads = {n: torch.full((96,), 7.0, dtype=c.pt, device="cuda")
             for n in ("pre_w", "pre_b", "post_w", "post_b")}
    if gate:
        grads["gate"] = torch.full_like(c.p["gate"], 7.0)
    c.m.moe_block_post_norm_bwd(c.desc, none, none, none, none, c.p, none, none, grads, c.ws)
    for n, t in grads.items():
        assert torch.count_nonzero(t) == 0, n


@pytest.mark.parametrize("gate", ["token", "full"])
@pytest.mark.parametrize("T,d", [(6, 256), (1300, 1024), (40, 77)])
def test_pre_norm_under_a_gated_descriptor(gate, T, d):
    """A block has one descriptor for both norms: the pre norm's calls have no
    gate, whatever it says of the post norm's."""
    plain, gated = Case(T=T, d=d, bias=True), Case(T=T, d=d, bias=True, gate=gate, act="sigmoid")
    res, dx, dres_in = plain.rows(plain.rt, 2.0), plain.rows(plain.at), plain.rows(plain.rt)
    got = []
    for c in (plain, gated):
        x, dres = c.empty(c.at), c.empty(c.rt)
        dw, db = torch.empty_like(plain.p["pre_w"]), torch.empty_like(plain.p["pre_b"])
        c.m.moe_block_pre_norm_fwd(c.desc, res, plain.p["pre_w"], plain.p["pre_b"], x)
        c.m.moe_block_pre_norm_bwd(c.desc, dx, res, plain.p["pre_w"], dres_in, dres, dw, db, c.ws,
                                   0.75)
        got.append((x, dres, dw, db))
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("gate", [None, "channel", "token", "full"])
@pytest.mark.parametrize("shape", [dict(T=40, d=264), dict(T=1300, d=1024), dict(T=40, d=77)], ids=str)
@pytest.mark.parametrize("next_norm", [True, False])
def test_without_a_post_norm_dy_does_not_depend_on_y(gate, shape, next_norm):
    """dy = b G D: what y holds, an Inf or NaN too, has no part in it."""
    c = Case(**shape, post=None, gate=gate, act="tanh" if gate else None)
    y, r, dres_in = c.rows(c.at), c.rows(c.rt), c.rows(c.rt)
    dx = c.rows(c.at) if next_norm else None

    def backward():
        dres, dy = c.empty(c.rt), c.empty(c.at)
        c.m.moe_block_post_norm_bwd(c.desc, dres_in, dx, r if next_norm else None, y, c.p, dres, dy,
                                    {}, c.ws, 0.75)
        return dres, dy

    clean = backward()
    y[3, 5], y[9, 0], y[20, c.d - 1], y[39] = float("inf"), float("-inf"), float("nan"), 1e30
    for a, b in zip(clean, backward()):
        assert torch.isfinite(a).all() and torch.equal(a, b)
