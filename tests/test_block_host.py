"""Host side of the residual block's norms and of the gradient lists, without a
GPU: calls whose arguments are in order reach the check of the workspace
behind them, what the binding says of a list's tensors, and how it is built."""
import ctypes
import os
import sysconfig

import pytest
import torch


@pytest.fixture(scope="module")
def m():
    from moe_expert_mlp_gb300.build import build_library
    build_library()
    import moe_expert_mlp_gb300 as m
    m.lib()
    return m


NULL, WORKSPACE = 1, 4
AT = 1 << 20            # an aligned address the host checks never read


def post_bwd(m, T, kind, gate, p=None):
    """Status of a post norm's backward with row tensors and gate at `p` and a
    workspace of no bytes."""
    L = m._lib
    desc = m.make_block_norm_desc(T, 64, post_norm="rms", gate=kind)
    r = L.moe_rows_t(p, 64)
    params = L.moe_block_params_t(AT, None, AT, None, L.moe_rows_t(gate, 64))
    grads = L.moe_block_params_t(AT, None, AT, None, L.moe_rows_t(gate, 64))
    return m.lib().moe_block_post_norm_bwd(
        ctypes.byref(desc), r, 1.0, r, r, r, ctypes.byref(params), r, r, ctypes.byref(grads), AT, 0,
        None)


@pytest.mark.parametrize("kind", ["token", "full"])
def test_no_tokens_need_no_gate_values(m, kind):
    assert post_bwd(m, 0, kind, None) == WORKSPACE     # every argument in order
    assert post_bwd(m, 0, kind, AT) == WORKSPACE
    assert post_bwd(m, 4, kind, AT, AT) == WORKSPACE
    assert post_bwd(m, 4, kind, None, AT) == NULL


def test_a_channel_gate_is_needed_without_tokens_too(m):
    assert post_bwd(m, 0, "channel", None) == NULL     # its gradient's parameters
    assert post_bwd(m, 0, "channel", AT) == WORKSPACE


def described(m, g):
    """The list's tensors and outs as its array has them."""
    return [(a.grad, a.out, a.rows, a.cols, a.ld, a.ld_out, a.dtype, a.out_dtype)
            for a in g.array[:len(g)]]


BASE = dict(whole=lambda b: b[:48], shorter=lambda b: b[:20], longer=lambda b: b[:],
            matrix=lambda b: b[:48].view(6, 8), rows=lambda b: b[:48].view(6, 8)[:, :5],
            rows_wider_apart=lambda b: b.view(6, 16)[:, :5], columns=lambda b: b[:48].view(6, 8).t(),
            every_other=lambda b: b[:48:2], other_type=lambda b: b.view(torch.bfloat16)[:48],
            other_type_as_long=lambda b: b.view(torch.bfloat16)[:96], nothing=lambda b: b[:0])


@pytest.mark.parametrize("before", list(BASE))
@pytest.mark.parametrize("after", list(BASE))
def test_a_tensor_changed_at_its_address_is_described_anew(m, monkeypatch, before, after):
    """A list's description is the one that a new list of the same tensors has,
    also where a tensor, or its out, changed under its address."""
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)     # described, not run
    a, b, still = torch.zeros(96), torch.zeros(96), torch.zeros(7)
    for outs in (False, True):
        t, o = BASE[before](a), BASE[before](b)
        g = m.GradList([still, t], [still, o] if outs else None)
        t.data, o.data = BASE[after](a), BASE[after](b)
        g.refresh(outs=True)
        assert described(m, g) == described(m, m.GradList([still, t], [still, o] if outs else None))


def test_a_changed_out_is_described_anew_when_it_is_written(m, monkeypatch):
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    t, wide = torch.zeros(6, 8), torch.zeros(6, 16)
    o = wide.view(-1)[:48].view(6, 8)
    g = m.GradList([t], [o])
    o.data = wide[:, :8]
    g.refresh(outs=True)
    assert described(m, g) == described(m, m.GradList([t], [o]))
    o.data = wide[:3, :8]
    g.refresh(outs=False)               # the norm reads no out
    with pytest.raises(ValueError):
        g.refresh(outs=True)            # another shape


def test_a_list_that_grew_is_described_anew(m, monkeypatch):
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    g = m.GradList([torch.zeros(3)])
    g.tensors.append(torch.zeros(5))
    g.refresh()
    assert [a.cols for a in g.array] == [3, 5]
    g = m.GradList([torch.zeros(3)], [torch.zeros(3)])
    g.tensors.append(torch.zeros(5))
    with pytest.raises(ValueError):
        g.refresh()


@pytest.mark.parametrize("compiler", ["false", "/nowhere/cc"])
def test_the_library_stands_without_the_binding(m, monkeypatch, tmp_path, capfd, compiler):
    """Where the binding cannot be compiled (no Python headers, no C compiler)
    the library still builds; the calls that need the binding raise, and an
    outdated one is not left to be loaded."""
    from moe_expert_mlp_gb300 import build
    L = m._lib
    at = tmp_path / "_binding.so"
    at.write_bytes(b"of another header")
    os.utime(at, (0, 0))
    monkeypatch.setattr(build, "BINDING", str(at))
    monkeypatch.setattr(L, "BINDING_PATH", str(at))
    monkeypatch.setattr(L, "_binding", None)
    monkeypatch.setenv("CC", compiler)
    assert build.build_library() == build.LIB
    assert "binding is not built" in capfd.readouterr().err
    assert list(tmp_path.iterdir()) == []
    with pytest.raises(m.MoeError):
        m.moe_block_pre_norm_fwd(m.make_block_norm_desc(4, 64), None, None, None, None)
    assert m.moe_fc1_padded_width(2880) == 2944            # the others do not need it


def test_the_binding_is_named_for_its_python(m):
    from moe_expert_mlp_gb300 import build
    assert build.BINDING == m._lib.BINDING_PATH
    assert build.BINDING.endswith("_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
    assert m._lib.binding().__file__ == build.BINDING


def test_two_gradients_are_not_clipped_into_the_same_memory(m, monkeypatch):
    """A gradient listed twice (a tied weight's) would be scaled by two blocks at
    once: refused before anything is enqueued.  Its norm may be taken."""
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    a, b, out = torch.zeros(3), torch.zeros(3), torch.zeros(3)
    norm = torch.zeros(1)
    for lst in ([a, b, a], m.GradList([a, b, a]), m.GradList([a, b], [out, out])):
        with pytest.raises(ValueError, match="same memory"):
            m.moe_clip_grads(lst, norm, 1.0)
    wide = torch.zeros(4, 8)
    for fine in (m.GradList([a, a], [b, out]), m.GradList([wide[:, :4], wide[:, 4:]]),
                 m.GradList([a[:0], a[:0], a])):
        assert fine.shared is None
    g = m.GradList([a, b])
    b.data = a                          # tied since
    with pytest.raises(ValueError, match="same memory"):
        m.moe_clip_grads(g, norm, 1.0)
