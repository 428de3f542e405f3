"""Host side of the residual block's norms and of the gradient lists, without a
GPU: calls whose arguments are in order reach the check of the workspace
behind them, and what the binding says of a list's tensors."""
import ctypes

import pytest


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
