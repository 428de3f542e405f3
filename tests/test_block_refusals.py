"""The residual block's norms and the gradient calls refuse bad arguments on
the host, before anything is enqueued: the C calls with a status, the binding
with ValueError."""
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


def rows(L, p=AT, ld=64):
    return L.moe_rows_t(p, ld)


def pre_fwd(m, desc, **over):
    L = m._lib
    a = dict(res=rows(L), w=AT, b=None, x=rows(L))
    a.update(over)
    return m.lib().moe_block_pre_norm_fwd(ctypes.byref(desc), a["res"], a["w"], a["b"], a["x"], None)


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), SHAPE), (dict(T=(1 << 30) + 1), SHAPE), (dict(d=0), SHAPE), (dict(d=16385), SHAPE),
    (dict(dtype=2), UNSUPPORTED), (dict(res_dtype=3), UNSUPPORTED),
    (dict(param_dtype=0), UNSUPPORTED), (dict(dtype=4, res_dtype=1), UNSUPPORTED),
    (dict(pre_norm=3), UNSUPPORTED), (dict(post_norm=-1), UNSUPPORTED), (dict(gate=4), UNSUPPORTED),
    (dict(gate_act=3), UNSUPPORTED), (dict(pre_eps=0.0), SHAPE), (dict(post_eps=-1.0), SHAPE),
    (dict(pre_eps=float("nan")), SHAPE), (dict(res_scale=float("inf")), SHAPE),
    (dict(branch_scale=float("nan")), SHAPE), (dict(pre_offset=float("inf")), SHAPE)])
def test_descriptor(m, change, status):
    desc = m.make_block_norm_desc(4, 64, post_norm="rms")
    for n, v in change.items():
        setattr(desc, n, v)
    size = ctypes.c_size_t(0)
    assert m.lib().moe_block_norm_workspace_size(ctypes.byref(desc), ctypes.byref(size)) == status
    assert pre_fwd(m, desc) == status


def test_pre_norm_arguments(m):
    L = m._lib
    desc = m.make_block_norm_desc(4, 64)
    assert m.lib().moe_block_pre_norm_fwd(None, rows(L), AT, None, rows(L), None) == NULL
    assert pre_fwd(m, m.make_block_norm_desc(4, 64, pre_norm=None)) == UNSUPPORTED
    assert pre_fwd(m, desc, res=rows(L, None)) == NULL
    assert pre_fwd(m, desc, x=rows(L, None)) == NULL
    assert pre_fwd(m, desc, x=rows(L, ld=63)) == SHAPE          # rows overlap
    assert pre_fwd(m, desc, res=rows(L, ld=-64)) == SHAPE
    assert pre_fwd(m, desc, res=rows(L, AT + 1)) == SHAPE       # not on an element
    assert pre_fwd(m, desc, w=AT + 1) == SHAPE
    # no tokens: nothing to do, nothing needed
    assert pre_fwd(m, m.make_block_norm_desc(0, 64), res=rows(L, None), x=rows(L, None)) == 0


def pre_bwd(m, desc, **over):
    L = m._lib
    a = dict(dx=rows(L), res=rows(L), dres_in=rows(L), scale=1.0, dres=rows(L), ws=AT,
             ws_bytes=1 << 30)
    a.update(over)
    return m.lib().moe_block_pre_norm_bwd(ctypes.byref(desc), a["dx"], a["res"], AT, a["dres_in"],
                                          a["scale"], a["dres"], AT, None, a["ws"], a["ws_bytes"],
                                          None)


def test_pre_norm_backward_arguments(m):
    L = m._lib
    desc = m.make_block_norm_desc(4, 64)
    for n in ("dx", "res", "dres"):
        assert pre_bwd(m, desc, **{n: rows(L, None)}) == NULL, n
    assert pre_bwd(m, desc, ws=None) == NULL
    assert pre_bwd(m, desc, ws=AT + 8) == SHAPE
    assert pre_bwd(m, desc, ws_bytes=m.moe_block_norm_workspace_size(desc) - 1) == WORKSPACE
    assert pre_bwd(m, desc, scale=float("nan")) == SHAPE
    assert pre_bwd(m, m.make_block_norm_desc(4, 64, pre_norm=None)) == UNSUPPORTED


def post_fwd(m, desc, **over):
    L = m._lib
    a = dict(res=rows(L), y=rows(L), gate=rows(L), res_out=rows(L), x=rows(L), routed=None,
             params=True)
    a.update(over)
    p = L.moe_block_params_t(AT, None, AT, None, a["gate"])
    r = None if a["routed"] is None else ctypes.byref(L.moe_routed_rows_t(*a["routed"]))
    return m.lib().moe_block_post_norm_fwd(
        ctypes.byref(desc), a["res"], a["y"], ctypes.byref(p) if a["params"] else None,
        a["res_out"], a["x"], r, None)


def test_post_norm_arguments(m):
    L = m._lib
    desc = m.make_block_norm_desc(4, 64, post_norm="rms", gate="token")
    for n in ("res", "y", "res_out", "gate"):
        assert post_fwd(m, desc, **{n: rows(L, None)}) == NULL, n
    assert post_fwd(m, desc, params=False) == NULL
    assert post_fwd(m, desc, gate=rows(L, ld=0)) == SHAPE
    assert post_fwd(m, desc, gate=rows(L, AT + 2, 1)) == SHAPE
    assert post_fwd(m, m.make_block_norm_desc(4, 64, pre_norm=None)) == UNSUPPORTED
    none = rows(L, None)
    assert post_fwd(m, desc, routed=(AT, AT, 0, 8, none)) == SHAPE
    assert post_fwd(m, desc, routed=(AT, AT, 33, 8, none)) == SHAPE
    assert post_fwd(m, desc, routed=(AT, AT, 2, -1, none)) == SHAPE
    assert post_fwd(m, desc, routed=(None, AT, 2, 8, none)) == NULL
    assert post_fwd(m, desc, routed=(AT, AT + 2, 2, 8, none)) == SHAPE


def test_post_norm_backward_arguments(m):
    L = m._lib
    desc = m.make_block_norm_desc(4, 64, post_norm="rms", gate="full")
    none = rows(L, None)

    def call(dres_in=rows(L), dx=rows(L), res_out=rows(L), y=rows(L), dy=rows(L), gate=rows(L),
             scale=1.0, d=desc):
        p = L.moe_block_params_t(AT, None, AT, None, gate)
        g = L.moe_block_params_t(AT, None, AT, None, none)
        return m.lib().moe_block_post_norm_bwd(
            ctypes.byref(d), dres_in, scale, dx, res_out, y, ctypes.byref(p), none, dy,
            ctypes.byref(g), AT, 1 << 30, None)

    assert call(dres_in=none, dx=none) == NULL          # no gradient at all
    assert call(res_out=none) == NULL                   # wanted by the next norm
    assert call(y=none) == NULL
    assert call(dy=none) == NULL
    assert call(gate=none) == NULL
    assert call(gate=rows(L, ld=32)) == SHAPE
    assert call(scale=float("inf")) == SHAPE
    assert call(d=m.make_block_norm_desc(4, 64, pre_norm=None, gate="full")) == UNSUPPORTED


def grad(L, **over):
    a = dict(grad=AT, out=AT, rows=1, cols=64, ld=64, ld_out=64, dtype=1, out_dtype=1)
    a.update(over)
    return L.moe_grad_t(*[a[n] for n, _ in L.moe_grad_t._fields_])


def test_gradient_list_arguments(m):
    L, lib = m._lib, m.lib()

    def norm(g=None, n=1, kind=0, out=AT, ws=AT, ws_bytes=1 << 20):
        a = (L.moe_grad_t * 1)(g if g is not None else grad(L))
        return lib.moe_grad_norm(a, n, kind, out, None, ws, ws_bytes, None)

    def clip(g=None, n=1, at=AT, most=1.0, eps=1e-6):
        a = (L.moe_grad_t * 1)(g if g is not None else grad(L))
        return lib.moe_clip_grads(a, n, at, most, eps, None)

    assert norm(n=-1) == SHAPE and clip(n=-1) == SHAPE
    assert norm(kind=2) == UNSUPPORTED
    assert norm(out=None) == NULL and norm(ws=None) == NULL and clip(at=None) == NULL
    assert norm(ws=AT + 4) == SHAPE and norm(out=AT + 2) == SHAPE
    assert norm(ws_bytes=m.moe_grad_norm_workspace_size(1) - 1) == WORKSPACE
    assert lib.moe_grad_norm(None, 1, 0, AT, None, AT, 1 << 20, None) == NULL
    assert lib.moe_clip_grads(None, 1, AT, 1.0, 0.0, None) == NULL
    for call in (norm, clip):
        assert call(grad(L, dtype=2)) == UNSUPPORTED
        assert call(grad(L, rows=-1)) == SHAPE
        assert call(grad(L, cols=-1)) == SHAPE
        assert call(grad(L, grad=None)) == NULL
        assert call(grad(L, grad=AT + 1)) == SHAPE
        assert call(grad(L, rows=2, ld=63)) == SHAPE
        assert call(grad(L, rows=1 << 30, cols=1 << 30, ld=1 << 30, ld_out=1 << 30)) == SHAPE
    assert clip(grad(L, out=None)) == NULL
    assert clip(grad(L, out_dtype=3)) == UNSUPPORTED
    assert clip(grad(L, out_dtype=4)) == UNSUPPORTED                # in place in another type
    assert clip(grad(L, rows=2, ld_out=80)) == UNSUPPORTED          # in place, other rows
    assert clip(grad(L, out=2 * AT, rows=2, ld_out=63)) == SHAPE
    assert clip(most=-1.0) == SHAPE and clip(most=float("nan")) == SHAPE
    assert clip(most=float("inf")) == SHAPE and clip(eps=-1.0) == SHAPE
    n = ctypes.c_size_t(0)
    assert lib.moe_grad_norm_workspace_size(-1, ctypes.byref(n)) == SHAPE
    assert lib.moe_grad_norm_workspace_size(1, None) == NULL


def test_binding_refuses_tensors_it_cannot_describe(m):
    desc = m.make_block_norm_desc(4, 64)
    on_cpu = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        m.moe_block_pre_norm_fwd(desc, on_cpu, None, None, on_cpu)
    with pytest.raises(ValueError):
        m.GradList([on_cpu])
    with pytest.raises(ValueError):
        m.GradList([], [on_cpu])
    with pytest.raises(KeyError):
        m.make_block_norm_desc(4, 64, pre_norm="batch")


def test_runs_of_a_tensor(m):
    runs = m._lib._runs
    t = torch.zeros(6, 10, 8)
    assert runs(t, t) == (1, 480, 480, 480)
    assert runs(t.transpose(0, 2), t.transpose(0, 2)) == (1, 480, 480, 480)
    assert runs(t[:, :, :3], t[:, :, :3]) == (60, 3, 8, 8)
    assert runs(t[:, 2:5], t[:, 2:5]) == (6, 24, 80, 80)
    assert runs(t[:, 2:5], torch.zeros(6, 3, 8)) == (6, 24, 80, 24)
    assert runs(t[0, :, 0], t[0, :, 0]) == (10, 1, 8, 8)
    assert runs(t[0, 0, :1], t[0, 0, :1]) == (1, 1, 1, 1)
    assert runs(t[:0], t[:0])[:2] == (1, 0)
    assert runs(torch.zeros(()), torch.zeros(())) == (1, 1, 1, 1)
    for bad in (t[:, 2:5, :3], torch.zeros(3).expand(5, 3), torch.zeros(1).expand(4)):
        with pytest.raises(ValueError):
            runs(bad, bad)
    with pytest.raises(ValueError):
        runs(t[0], torch.zeros(8, 10).t())            # another memory order
