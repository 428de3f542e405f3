"""A residual block's whole training step with the router's losses and the
experts' orthogonalised updates: each stage against the oracle applied to the
stage's own stored inputs, two steps with a momentum in a CUDA graph, and that a
layer without them is what it was.

Bounds: those of test_gpu_router_loss.py and test_gpu_orthogonalize.py."""
import numpy as np
import pytest
import torch

import oracle.training_oracle as O
from tests import harness as H
from tests.test_gpu_block_norm import f64
from tests.test_gpu_orthogonalize import check as check_updates
from tests.test_gpu_router_loss import check_backward, check_forward
from workloads import WORKLOADS, make_inputs, scaled

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

WL = scaled(WORKLOADS["bf16_t4096_e64"], T=330, E=8, k=3, d=320, F=160)
SMALL = scaled(WORKLOADS["tiny_t256_e8"], T=200, d=128, F=96)
BALANCE, Z, S = 0.02, 1e-3, 3


def make(wl, dtype="bf16", losses=True, **kw):
    import moe_expert_mlp_gb300 as m
    inp = make_inputs(wl)
    if losses:
        kw = dict(kw, balance_coef=BALANCE, z_coef=Z, sequences=S)
    layer = H.make_layer(wl, dtype=dtype, **kw)
    w = [H.bits_to_dev(inp[n]) for n in ("w1", "w2")]
    if dtype == "fp32":
        w = [t.float() for t in w]
    layer.load_weights(w[0], None, w[1], None)
    block = m.MoEResidualBlock(layer)
    g = torch.Generator().manual_seed(3)
    res = torch.randn(wl.T, wl.d, generator=g).to(layer.act_dtype).cuda()
    dres = (0.1 * torch.randn(wl.T, wl.d, generator=g)).to(layer.act_dtype).cuda()
    logits = torch.from_numpy(inp["logits"]).cuda()
    bias = torch.from_numpy(inp["bias"]).cuda() if inp["bias"] is not None else None
    mask = (torch.rand(wl.T, generator=g) > 0.2).cuda()
    offsets = torch.tensor([0, wl.T // 3, wl.T // 2, wl.T - 7], dtype=torch.int32).cuda()
    return m, block, res, logits, bias, dres, mask, offsets


def check_router(layer, logits, mask, offsets, dloss):
    T = layer.T
    idx = layer.topk_idx[:T].cpu().numpy()
    got = dict(counts=layer.loss_counts.cpu().numpy(), tokens=layer.loss_tokens.cpu().numpy(),
               probs=layer.loss_probs.cpu().numpy(), loss=layer.router_loss.cpu().numpy())
    l32, mk, off = logits.cpu().numpy(), mask.cpu().numpy(), offsets.cpu().numpy()
    check_forward(l32, idx, S, BALANCE, Z, mk, off, got)
    routed = (layer.dw[:T].cpu().numpy(), layer.topk_w[:T].cpu().numpy(), idx)
    check_backward(l32, layer.k, S, BALANCE, Z, mk, off, got, f64(layer.dlogits[:T]), dloss, routed)


@pytest.mark.parametrize("wl,dtype", [(WL, "bf16"), (SMALL, "fp32"), (SMALL, "mxfp8")])
def test_stages_match_oracle(wl, dtype):
    m, block, res, logits, bias, dres, mask, offsets = make(wl, dtype)
    layer = block.layer
    updates = block.orthogonal_updates(momentum=0.9, dampening=0.1, nesterov=True)
    dloss = torch.full((1,), 2.5, device="cuda")
    for _ in range(2):
        before = [f64(t) for t in updates.momenta]
        block.step(res, logits, bias, dres, max_norm=0.05, mask=mask, seq_offsets=offsets,
                   dloss=dloss)
        torch.cuda.synchronize()
        assert m.moe_read_device_status() == 0
        check_router(layer, logits, mask, offsets, 2.5)
        for g, m0, out, m1 in zip((layer.dw1p, layer.dw2), before, updates.outs, updates.momenta):
            rows, cols = g.shape[1:]
            check_updates(f64(g), m0, f64(out), f64(m1), momentum=0.9, dampening=0.1, nesterov=True,
                          scale=np.float32(0.2 * np.sqrt(max(rows, cols))))
    # the packed FC1's padding rows have no gradient and get no update
    pad = torch.ones(2 * layer.Fp, dtype=torch.bool)
    for block_of in range(layer.Fp // 128):
        real = min(128, layer.F - 128 * block_of)
        for half in (0, 128):
            pad[256 * block_of + half:256 * block_of + half + real] = False
    assert not updates.outs[0][:, pad.cuda()].any()


def test_two_steps_replay_in_a_cuda_graph():
    m, block, res, logits, bias, dres, mask, offsets = make(WL)
    updates = block.orthogonal_updates(momentum=0.95)
    args = dict(max_norm=0.05, mask=mask, seq_offsets=offsets)
    for _ in range(2):
        block.step(res, logits, bias, dres, **args)
    torch.cuda.synchronize()
    want = [t.clone() for t in updates.outs + updates.momenta + [block.layer.dlogits,
                                                                block.layer.router_loss]]
    for t in updates.momenta:
        t.zero_()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        block.step(res, logits, bias, dres, stream=s, **args)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert m.moe_read_device_status() == 0
    got = updates.outs + updates.momenta + [block.layer.dlogits, block.layer.router_loss]
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_a_layer_without_losses_is_what_it_was():
    m, block, res, logits, bias, dres, mask, offsets = make(WL, losses=False)
    layer = block.layer
    block.step(res, logits, bias, dres)
    plain = torch.empty_like(layer.dlogits)
    m.moe_route_bwd(layer.desc, layer.dw, layer.topk_w, layer.topk_idx, plain)
    assert torch.equal(plain, layer.dlogits) and block.updates is None
    with pytest.raises(ValueError, match="coefficients"):
        layer.route(block.x, logits, bias, mask=mask)


def test_fused_routing_needs_the_logits_for_the_losses():
    m, block, res, logits, bias, dres, mask, offsets = make(WL)
    layer = block.layer
    x = block.forward_norm(res)
    w_r = (0.05 * torch.randn(WL.E, WL.d, generator=torch.Generator().manual_seed(1))).to(
        torch.bfloat16).cuda()
    with pytest.raises(ValueError, match="logits_out"):
        layer.route_fused(x, w_r, bias)
    out = torch.zeros(WL.T, WL.E, device="cuda")
    layer.route_fused(x, w_r, bias, out, mask=mask, seq_offsets=offsets)
    layer.mlp_forward()
    layer.out.zero_()
    m._lib.moe_unpermute_combine(layer.desc, layer.y, layer.row_of, layer.topk_w, layer.out)
    layer.backward(dres)
    torch.cuda.synchronize()
    check_router(layer, out, mask, offsets, 1.0)


def test_updates_refuse_what_they_cannot_read():
    import moe_expert_mlp_gb300 as m
    with pytest.raises(ValueError, match="gradient 1"):
        m.OrthogonalUpdates([torch.zeros(2, 3, 4, device="cuda"), torch.zeros(7, device="cuda")])
    with pytest.raises(ValueError, match="gradient 0"):
        m.OrthogonalUpdates([torch.zeros(3, 4, device="cuda", dtype=torch.float16)])
    u = m.OrthogonalUpdates([torch.zeros(3, 4, device="cuda")], momentum=0.0, scale=0.5)
    assert u.momenta == [None] and not u.step()[0].any()
    assert m.OrthogonalUpdates([]).step() == []
