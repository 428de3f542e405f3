"""MoEResidualBlock on the GPU: every stage against the oracle applied to the
stage's own stored inputs, the whole step in a CUDA graph, and clipping.

Bounds: the norms' as in test_gpu_block_norm.py; the layer's are its own
(harness)."""
import numpy as np
import pytest
import torch

import oracle
import oracle.block_oracle as B
from tests import harness as H
from tests.test_gpu_block_norm import check, f64
from workloads import WORKLOADS, make_inputs, scaled

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

WL = scaled(WORKLOADS["bf16_t4096_e64"], T=330, E=8, k=3, d=320, F=160)
WLB = scaled(WORKLOADS["gptoss_t16384_e32"], T=200, E=6, k=2, d=192, F=96)


def make(wl, dtype="bf16", seed=0, **kw):
    import moe_expert_mlp_gb300 as m
    inp = make_inputs(wl)
    layer = H.make_layer(wl, dtype=dtype)
    H.load_layer_weights(layer, inp)
    block = m.MoEResidualBlock(layer, **kw)
    g = torch.Generator().manual_seed(seed)
    for n, p in block.params.items():
        p.add_((0.2 * torch.randn(p.shape, generator=g)).to(p.dtype).cuda())
    rt = block.res_out.dtype
    res = (2 * torch.randn(wl.T, wl.d, generator=g)).to(rt).cuda()
    dres = (0.1 * torch.randn(wl.T, wl.d, generator=g)).to(rt).cuda()
    logits = torch.from_numpy(inp["logits"]).cuda()
    bias = torch.from_numpy(inp["bias"]).cuda() if inp["bias"] is not None else None
    gate = torch.randn(wl.T, generator=g).cuda() if kw.get("gate") == "token" else None
    return m, inp, block, res, logits, bias, dres, gate


CASES = {
    "rms_channel": (WL, dict()),
    "layer_bias_res32": (WL, dict(pre_norm="layer", post_norm="layer", bias=True, res_dtype="fp32",
                                  res_scale=0.75, branch_scale=0.5)),
    "token_sigmoid_biased_experts": (WLB, dict(gate="token", gate_act="sigmoid", offset=1.0)),
    "no_post_norm": (WL, dict(post_norm=None, gate="channel", gate_act="tanh", branch_scale=0.25)),
}


@pytest.mark.parametrize("name", list(CASES))
def test_stages_match_oracle(name):
    wl, kw = CASES[name]
    m, inp, block, res, logits, bias, dres, gate = make(wl, **kw)
    layer = block.layer
    block.step(res, logits, bias, dres, gate=gate)
    torch.cuda.synchronize()
    assert m.moe_read_device_status() == 0
    T = wl.T
    q = {n: f64(p) for n, p in block.params.items()}
    q["gate"] = f64(gate) if gate is not None else q.get("gate")
    kind = kw.get("gate", "channel")
    offset, a, b = kw.get("offset", 0.0), kw.get("res_scale", 1.0), kw.get("branch_scale", 1.0)
    pre = B.NormSpec(kw.get("pre_norm", "rms"), 1e-6, offset)
    post = B.NormSpec(kw.get("post_norm", "rms"), 1e-6, offset)
    check("x", block.x, *B.norm_fwd(f64(res), pre, q["pre_w"], q.get("pre_b")), 128)
    # the layer on the stored x
    p = H.glu_params(wl)
    W1, b1, W2, b2 = H.oracle_weights(inp)
    fwd = oracle.moe_forward(f64(block.x), inp["logits"], inp["bias"], W1, b1, W2, b2, wl.k, p,
                             align=128)
    H.assert_close("out", H.to_np(layer.out)[:T], fwd["out"])
    # the post norm on the stored expert rows
    y, mag_y = B.combine_rows(f64(layer.y), layer.row_of.cpu().numpy(), layer.topk_w.cpu().numpy())
    check("combined", layer.out, y, mag_y, 64)
    act = kw.get("gate_act")
    r, mag = B.post_fwd(f64(res), y, mag_y, post, q.get("post_w"), q.get("post_b"), q["gate"], kind,
                        act, a, b)
    check("res_out", block.res_out, r, mag, 192)
    # backward of the post norm on the stored combined rows
    D = f64(dres)
    ref = B.post_bwd(D, np.abs(D), f64(layer.out), post, q.get("post_w"), q.get("post_b"),
                     q["gate"], kind, act, b)
    check("dout", block.dout, *ref["dy"], 256)
    check("dgate", block.grads["gate"], *ref["gate"], 256 + 192 + T)
    if post.kind is not None:
        check("dpost_w", block.grads["post_w"], *ref["dw"], 256 + 192 + T)
    # the layer's backward on the stored dout
    bwd = oracle.moe_backward(fwd, f64(block.dout), W1, W2, p)
    H.assert_close("dx", H.to_np(layer.dx)[:T], bwd["dx"])
    H.assert_close("dW2", H.to_np(layer.dw2), bwd["dW2"])
    # and the pre norm's on the stored dx
    (D, mag), dw, db = B.join_grads(f64(dres), f64(layer.dx), f64(res), pre, q["pre_w"], a)
    check("dres", block.dres, D, mag, 128)
    check("dpre_w", block.grads["pre_w"], *dw, 128 + 192 + T)
    if "pre_b" in block.grads:
        check("dpre_b", block.grads["pre_b"], *db, 128 + 192 + T)


@pytest.mark.parametrize("dtype", ["mxfp8", "fp32"])
def test_other_operand_types_run(dtype):
    """The block around an MXFP8 and an fp32 layer: finite, and the norms on
    the stored tensors exact."""
    wl = scaled(WORKLOADS["tiny_t256_e8"], T=200, d=256, F=128)
    import moe_expert_mlp_gb300 as m
    inp = make_inputs(wl)
    layer = H.make_layer(wl, dtype=dtype)
    bf = [H.bits_to_dev(inp[n]) for n in ("w1", "w2")]
    if dtype == "fp32":
        bf = [t.float() for t in bf]
    layer.load_weights(bf[0], None, bf[1], None)
    block = m.MoEResidualBlock(layer)
    g = torch.Generator().manual_seed(1)
    res = torch.randn(wl.T, wl.d, generator=g).to(layer.act_dtype).cuda()
    dres = torch.randn(wl.T, wl.d, generator=g).to(layer.act_dtype).cuda()
    block.step(res, torch.from_numpy(inp["logits"]).cuda(), None, dres, max_norm=1.0)
    torch.cuda.synchronize()
    assert m.moe_read_device_status() == 0
    spec = B.NormSpec("rms", 1e-6)
    check("x", block.x, *B.norm_fwd(f64(res), spec, f64(block.params["pre_w"])), 128)
    (D, mag), _, _ = B.join_grads(f64(dres), f64(layer.dx), f64(res), spec,
                                  f64(block.params["pre_w"]))
    check("dres", block.dres, D, mag, 128)
    total, _ = B.grad_norm([f64(t) for t in block.gradients.tensors])
    assert total <= 1.0 + 2.0 ** -8            # clipped values, rounded to their type


def test_clipping_of_the_block():
    m, _, block, res, logits, bias, dres, _ = make(WL)
    block.step(res, logits, bias, dres)
    before = [t.clone() for t in block.gradients.tensors]
    total, each = B.grad_norm([f64(t) for t in before])
    block.clip_gradients(0.5 * total)
    assert abs(float(block.norm) - total) <= 18 * 2.0 ** -24 * total
    assert np.all(np.abs(f64(block.norms) - each) <= 18 * 2.0 ** -24 * each)
    f = B.clip_factor(float(block.norm), np.float32(0.5 * total), 1e-6)
    for t, o in zip(block.gradients.tensors, before):
        ref = f64(o) * f
        assert np.all(np.abs(f64(t) - ref) <= (2.0 ** -8 + 4 * 2.0 ** -24) * np.abs(ref) + 1e-40)


def test_whole_step_replays_in_a_cuda_graph():
    m, _, block, res, logits, bias, dres, _ = make(WL)
    block.step(res, logits, bias, dres, max_norm=0.1)
    torch.cuda.synchronize()
    names = ("res_out", "dres", "norm")
    want = {n: getattr(block, n).clone() for n in names}
    grads = [t.clone() for t in block.gradients.tensors]
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        block.step(res, logits, bias, dres, max_norm=0.1, stream=s)
    for n in names:
        getattr(block, n).zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert m.moe_read_device_status() == 0
    for n in names:
        assert torch.equal(getattr(block, n), want[n]), n
    for a, b in zip(block.gradients.tensors, grads):
        assert torch.equal(a, b)


def test_refusals():
    import moe_expert_mlp_gb300 as m
    direct = H.make_layer(scaled(WORKLOADS["dsv3_r16384_e32"], R=300, E=4, d=128, F=64), capacity=1024)
    with pytest.raises(ValueError):
        m.MoEResidualBlock(direct)
    m, _, block, res, logits, bias, dres, gate = make(WLB, gate="token")
    with pytest.raises(ValueError):
        block.forward(res, logits, bias)
    with pytest.raises(ValueError):
        m.MoEResidualBlock(block.layer, gate="full")
    with pytest.raises(ValueError):
        block.forward(res[:, :64], logits, bias, gate=gate)
    with pytest.raises(ValueError):
        block.forward(res.float(), logits, bias, gate=gate)
