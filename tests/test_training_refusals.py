"""The router's losses and orthogonalised updates refuse bad arguments on the
host, before anything is enqueued: the C calls with a status, the binding with
ValueError."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def m():
    from moe_expert_mlp_gb300.build import build_library
    build_library()
    import moe_expert_mlp_gb300 as m
    m.lib()
    return m


NULL, SHAPE, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4
AT = 1 << 20            # an aligned address the host checks never read
BIG = 1 << 40


# ------------------------------------------------------- router's losses
def loss_fwd(m, desc, **over):
    a = dict(logits=AT, idx=AT, mask=None, offsets=AT, counts=AT, tokens=AT, probs=AT, loss=AT,
             ws=AT, ws_bytes=BIG)
    a.update(over)
    return m.lib().moe_router_loss_fwd(
        ctypes.byref(desc) if desc is not None else None, a["logits"], a["idx"], a["mask"],
        a["offsets"], a["counts"], a["tokens"], a["probs"], a["loss"], a["ws"], a["ws_bytes"], None)


def loss_bwd(m, desc, **over):
    a = dict(logits=AT, mask=None, offsets=AT, counts=AT, tokens=AT, dloss=None, dw=None, w=None,
             idx=None, dlogits=AT)
    a.update(over)
    return m.lib().moe_router_loss_bwd(
        ctypes.byref(desc) if desc is not None else None, a["logits"], a["mask"], a["offsets"],
        a["counts"], a["tokens"], a["dloss"], a["dw"], a["w"], a["idx"], a["dlogits"], None)


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), SHAPE), (dict(T=(1 << 28) + 1), SHAPE), (dict(E=0), SHAPE), (dict(E=257), SHAPE),
    (dict(k=0), SHAPE), (dict(k=9), SHAPE), (dict(E=64, k=33), SHAPE), (dict(sequences=0), SHAPE),
    (dict(sequences=65536), SHAPE), (dict(balance_coef=float("nan")), SHAPE),
    (dict(z_coef=float("inf")), SHAPE)])
def test_router_loss_descriptor(m, change, status):
    desc = m.make_router_loss_desc(16, 8, 2, 2)
    for n, v in change.items():
        setattr(desc, n, v)
    size = ctypes.c_size_t(0)
    assert m.lib().moe_router_loss_workspace_size(ctypes.byref(desc), ctypes.byref(size)) == status
    assert loss_fwd(m, desc) == status and loss_bwd(m, desc) == status


def test_router_loss_arguments(m):
    desc = m.make_router_loss_desc(16, 8, 2, 2)
    size = ctypes.c_size_t(0)
    assert m.lib().moe_router_loss_workspace_size(None, ctypes.byref(size)) == NULL
    assert m.lib().moe_router_loss_workspace_size(ctypes.byref(desc), None) == NULL
    assert loss_fwd(m, None) == NULL and loss_bwd(m, None) == NULL
    for n in ("logits", "idx", "offsets", "counts", "tokens", "probs", "loss", "ws"):
        assert loss_fwd(m, desc, **{n: None}) == NULL, n
        assert loss_fwd(m, desc, **{n: AT + 2}) == SHAPE, n
    assert loss_fwd(m, desc, ws=AT + 8) == SHAPE
    need = m.moe_router_loss_workspace_size(desc)
    assert loss_fwd(m, desc, ws_bytes=need - 1) == WORKSPACE
    for n in ("logits", "offsets", "counts", "tokens", "dlogits"):
        assert loss_bwd(m, desc, **{n: None}) == NULL, n
        assert loss_bwd(m, desc, **{n: AT + 2}) == SHAPE, n
    assert loss_bwd(m, desc, dloss=AT + 2) == SHAPE
    assert loss_bwd(m, desc, dw=AT) == NULL
    assert loss_bwd(m, desc, dw=AT, w=AT) == NULL
    assert loss_bwd(m, desc, dw=AT, w=AT + 1, idx=AT) == SHAPE
    assert loss_bwd(m, desc, dw=AT, w=AT, idx=AT + 1) == SHAPE


def test_binding_refuses_host_tensors_and_other_descriptors(m):
    desc = m.make_router_loss_desc(4, 8, 2)
    f, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    out = [torch.zeros(1, 8, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
           torch.zeros(1, 8), torch.zeros(3)]
    ws = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(ValueError):
        m.moe_router_loss_fwd(desc, f, i, None, None, *out, ws)
    with pytest.raises(ValueError):
        m.moe_router_loss_bwd(desc, f, None, None, out[0], out[1], None, None, f)
    with pytest.raises(ValueError, match="routed"):
        m.moe_router_loss_bwd(desc, f, None, None, out[0], out[1], None, {"dw": f}, f)
    other = m.make_orthogonalize_desc(1, 4, 8)
    with pytest.raises(ValueError, match="descriptor"):
        m.moe_router_loss_fwd(other, f, i, None, None, *out, ws)
    with pytest.raises(ValueError, match="descriptor"):
        m.moe_orthogonalize(desc, f, f, ws)
    with pytest.raises(ValueError):
        m.moe_orthogonalize(other, f, f, ws)


# ------------------------------------------------- orthogonalised updates
def mats(m, p=AT, ld=64, plane=64 * 32):
    return m._lib.moe_matrices_t(p, ld, plane)


def ortho(m, desc, **over):
    a = dict(grad=mats(m), mom=mats(m, None, 0, 0), mom_out=mats(m, None, 0, 0), out=mats(m), ws=AT,
             ws_bytes=BIG)
    a.update(over)
    return m.lib().moe_orthogonalize(ctypes.byref(desc) if desc is not None else None, a["grad"],
                                     a["mom"], a["mom_out"], a["out"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("change,status", [
    (dict(batch=-1), SHAPE), (dict(batch=65536), SHAPE), (dict(rows=0), SHAPE),
    (dict(rows=16385), SHAPE), (dict(cols=0), SHAPE), (dict(cols=16385), SHAPE),
    (dict(steps=0), SHAPE), (dict(steps=17), SHAPE), (dict(grad_dtype=2), UNSUPPORTED),
    (dict(eps=0.0), SHAPE), (dict(eps=float("inf")), SHAPE), (dict(eps=-1.0), SHAPE),
    (dict(a=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE),
    (dict(momentum=float("nan")), SHAPE), (dict(dampening=float("inf")), SHAPE),
    # a singular value in [0,1] could reach 2
    (dict(a=2.0, b=0.0, c=0.0), UNSUPPORTED), (dict(a=1.5, b=0.0, c=0.0, steps=2), UNSUPPORTED),
    (dict(a=6.0, b=-10.0, c=5.0), UNSUPPORTED), (dict(a=-3.0, b=0.5, c=0.4), UNSUPPORTED),
    # B could pass 16
    (dict(a=2.0, b=-17.0, c=15.0), UNSUPPORTED), (dict(a=1.0, b=-12.0, c=11.5), UNSUPPORTED)])
def test_orthogonalize_descriptor(m, change, status):
    desc = m.make_orthogonalize_desc(2, 32, 64)
    for n, v in change.items():
        setattr(desc, n, v)
    size = ctypes.c_size_t(0)
    assert m.lib().moe_orthogonalize_workspace_size(ctypes.byref(desc), ctypes.byref(size)) == status
    assert ortho(m, desc) == status


@pytest.mark.parametrize("coefficients,steps", [((3.4445, -4.7750, 2.0315), 16), ((1.5, -0.5, 0.0), 16),
                                                ((1.875, -1.25, 0.375), 16), ((1.9, 0.0, 0.0), 1),
                                                ((2.0, -1.5, 0.5), 16)])
def test_coefficients_that_hold(m, coefficients, steps):
    assert m.moe_orthogonalize_workspace_size(
        m.make_orthogonalize_desc(2, 32, 64, coefficients=coefficients, steps=steps)) > 0


def test_orthogonalize_arguments(m):
    desc = m.make_orthogonalize_desc(2, 32, 64)
    size = ctypes.c_size_t(0)
    assert m.lib().moe_orthogonalize_workspace_size(None, ctypes.byref(size)) == NULL
    assert m.lib().moe_orthogonalize_workspace_size(ctypes.byref(desc), None) == NULL
    assert ortho(m, None) == NULL
    for n in ("grad", "out"):
        assert ortho(m, desc, **{n: mats(m, None)}) == NULL, n
        assert ortho(m, desc, **{n: mats(m, AT + 1)}) == SHAPE, n
        assert ortho(m, desc, **{n: mats(m, ld=63)}) == SHAPE, n
        assert ortho(m, desc, **{n: mats(m, ld=-64)}) == SHAPE, n
    assert ortho(m, desc, out=mats(m, plane=64 * 32 - 1)) == SHAPE       # matrices overlap
    assert ortho(m, desc, ws=None) == NULL
    assert ortho(m, desc, ws=AT + 128) == SHAPE
    need = m.moe_orthogonalize_workspace_size(desc)
    assert ortho(m, desc, ws_bytes=need - 1) == WORKSPACE
    with_momentum = m.make_orthogonalize_desc(2, 32, 64, momentum=0.9)
    assert ortho(m, with_momentum) == NULL
    assert ortho(m, with_momentum, mom=mats(m)) == NULL
    assert ortho(m, with_momentum, mom_out=mats(m)) == NULL
    assert ortho(m, with_momentum, mom=mats(m, AT + 2), mom_out=mats(m)) == SHAPE
    assert ortho(m, with_momentum, mom=mats(m), mom_out=mats(m, plane=64)) == SHAPE
    assert ortho(m, desc, mom=mats(m)) == NULL                          # kept, but not where to
