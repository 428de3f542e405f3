"""MoEResidualBlock on the GPU: around an NVFP4 layer, with as many experts a
token as the framework's layers have, and with a router that reads the block's
own x.  Bounds: the norms' as in test_gpu_block_norm.py."""
import pytest
import torch

import oracle.block_oracle as B
from tests import harness as H
from tests.test_gpu_block_layer import WL, make
from tests.test_gpu_block_norm import check, f64
from workloads import WORKLOADS, make_inputs, scaled

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def check_stages(block, res, dres, T):
    """The norms on the tensors that the block stored."""
    layer, spec = block.layer, B.NormSpec("rms", 1e-6)
    q = {n: f64(p) for n, p in block.params.items()}
    check("x", block.x, *B.norm_fwd(f64(res), spec, q["pre_w"]), 128)
    y, mag_y = B.combine_rows(f64(layer.y), layer.row_of.cpu().numpy(), layer.topk_w.cpu().numpy())
    check("combined", layer.out, y, mag_y, 64)
    check("res_out", block.res_out, *B.post_fwd(f64(res), y, mag_y, spec, q["post_w"], None,
                                                q["gate"], "channel"), 192)
    D = f64(dres)
    ref = B.post_bwd(D, abs(D), f64(layer.out), spec, q["post_w"], None, q["gate"], "channel")
    check("dout", block.dout, *ref["dy"], 256)
    (D, mag), dw, _ = B.join_grads(D, f64(layer.dx), f64(res), spec, q["pre_w"])
    check("dres", block.dres, D, mag, 128)
    check("dpre_w", block.grads["pre_w"], *dw, 128 + 192 + T)


@pytest.mark.parametrize("dtype", ["nvfp4", "mxfp8", "bf16"])
@pytest.mark.parametrize("k", [6, 8])
def test_many_experts_a_token(dtype, k):
    import moe_expert_mlp_gb300 as m
    wl = scaled(WORKLOADS["tiny_t256_e8"], T=200, d=256, F=128, k=k)
    inp = make_inputs(wl)
    layer = H.make_layer(wl, dtype=dtype)
    H.load_layer_weights(layer, inp)
    block = m.MoEResidualBlock(layer)
    g = torch.Generator().manual_seed(2)
    res = torch.randn(wl.T, wl.d, generator=g).to(layer.act_dtype).cuda()
    dres = torch.randn(wl.T, wl.d, generator=g).to(layer.act_dtype).cuda()
    block.step(res, torch.from_numpy(inp["logits"]).cuda(), None, dres)
    torch.cuda.synchronize()
    assert m.moe_read_device_status() == 0
    check_stages(block, res, dres, wl.T)
    block.clip_gradients(1.0)
    total, _ = B.grad_norm([f64(t) for t in block.gradients.tensors])
    assert total <= 1.0 + 2.0 ** -8            # clipped values, rounded to their type


def test_a_router_that_reads_the_blocks_x():
    """x from forward_norm, logits from it, forward; the router's gradient joins
    layer.dx between backward_branch and backward_norm."""
    m, inp, block, res, logits, bias, dres, _ = make(WL)
    layer = block.layer
    g = torch.Generator().manual_seed(3)
    w_router = (0.05 * torch.randn(WL.E, WL.d, generator=g)).cuda()
    x = block.forward_norm(res)
    first = x.clone()
    own = x.float() @ w_router.t()
    block.forward(res, own, bias)
    assert torch.equal(block.x, first)
    block.backward_branch(dres)
    alone = layer.dx.clone()
    layer.dx.add_((layer.dlogits[:WL.T] @ w_router).to(layer.dx.dtype))
    assert not torch.equal(alone, layer.dx)
    block.backward_norm(dres)
    torch.cuda.synchronize()
    assert m.moe_read_device_status() == 0
    check_stages(block, res, dres, WL.T)
