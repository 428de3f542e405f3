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
