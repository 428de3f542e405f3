"""One residual block around a routed-expert MLP layer on one GPU: pre norm,
the layer, post norm with gate and scaled residual, their backward, the clipping
of the block's gradients and the updates they give the experts.

    x     = N1(res)
    out   = MoE(x)                         (MoEExpertMLP, combined tokens)
    res'  = res_scale*res + branch_scale * G (*) N2(out)

Like the layer, the block allocates all its buffers once and issues a fixed
sequence of C-ABI calls on one stream, so a whole step can be captured in one
CUDA graph.  The expert rows are combined inside the post norm's kernel.
"""
from __future__ import annotations

import torch

from . import _lib as L
from .updates import OrthogonalUpdates


class MoEResidualBlock:
    """layer: a routed MoEExpertMLP (T > 0).  Norms "rms" or "layer" (post_norm
    also None), gate None, "channel" or "token" (a value per token, given to
    forward) with gate_act None, "sigmoid" or "tanh"; res_dtype "bf16" or
    "fp32" for the residual stream.  Parameters start at the identity: weights
    (plus offset) one, biases zero, channel gate one."""

    def __init__(self, layer, pre_norm="rms", post_norm="rms", eps=1e-6, offset=0.0, bias=False,
                 gate="channel", gate_act=None, res_scale=1.0, branch_scale=1.0, res_dtype=None):
        if layer.T < 1:
            raise ValueError("the block needs a routed layer (T > 0)")
        if gate not in (None, "none", "channel", "token"):
            raise ValueError(f"gate {gate!r}: expected None, 'channel' or 'token'")
        dtype = "fp32" if layer.f32 else "bf16"
        self.layer = layer
        T, d, dev = layer.T, layer.d, layer.w2.device
        self.desc = L.make_block_norm_desc(
            T, d, dtype=dtype, res_dtype=res_dtype, pre_norm=pre_norm, post_norm=post_norm,
            pre_eps=eps, post_eps=eps, pre_offset=offset, post_offset=offset, gate=gate,
            gate_act=gate_act, res_scale=res_scale, branch_scale=branch_scale)
        self.res_scale = res_scale
        at = layer.act_dtype
        rt = torch.float32 if self.desc.res_dtype == L.MOE_DTYPE_FP32 else torch.bfloat16

        def vector(value):
            return torch.full((d,), value, dtype=at, device=dev)

        def rows(dtype):
            return torch.zeros((T, d), dtype=dtype, device=dev)

        self.params = {"pre_w": vector(1.0 - offset)}
        if bias:
            self.params["pre_b"] = vector(0.0)
        if post_norm not in (None, "none"):
            self.params["post_w"] = vector(1.0 - offset)
            if bias:
                self.params["post_b"] = vector(0.0)
        if gate == "channel":
            self.params["gate"] = vector(1.0)
        self.grads = {n: torch.zeros_like(p) for n, p in self.params.items()}
        self.token_gate = gate == "token"
        if self.token_gate:            # the gate is an input: its gradient per token
            self.grads["gate"] = torch.zeros(T, dtype=torch.float32, device=dev)
        self.gate = None
        self.x, self.res, self.res_out = rows(at), None, rows(rt)
        self.dout, self.dres = rows(at), rows(rt)
        self.ws = torch.empty(L.moe_block_norm_workspace_size(self.desc), dtype=torch.uint8,
                              device=dev)
        # the gradients that are the parameters': the token gate's is an input's
        mine = [g for n, g in self.grads.items() if not (self.token_gate and n == "gate")]
        self.gradients = L.GradList(
            [g for g in (layer.dw1p, layer.dw2, layer.db1p, layer.db2) if g is not None] + mine)
        n = len(self.gradients)
        self.norm = torch.zeros(1, dtype=torch.float32, device=dev)
        self.norms = torch.zeros(n, dtype=torch.float32, device=dev)
        self.norm_ws = torch.empty(L.moe_grad_norm_workspace_size(n), dtype=torch.uint8, device=dev)
        self.updates = None            # the experts', see orthogonal_updates

    def orthogonal_updates(self, padding=True, **kw):
        """From now on step() ends with the orthogonalised updates of the experts'
        weights, self.updates.outs for layer.w1p and layer.w2 (their clipped
        gradients' matrices, one an expert: gate and linear half of FC1 together;
        the packed FC1's padding rows stay zero); kw: as OrthogonalUpdates.  The scale
        goes by the packed rows, 2*Fp, which with F not a multiple of 128 makes FC1's
        update larger by up to sqrt(Fp/F); with padding=False by the weights' own."""
        layer = self.layer
        if not padding:
            kw["sizes"] = [(2 * layer.F if layer.gated else layer.F, layer.d), (layer.d, layer.F)]
        self.updates = OrthogonalUpdates([layer.dw1p, layer.dw2], **kw)
        return self.updates

    def forward_norm(self, res, stream=None):
        """x = N1(res), the layer's input (and the router's)."""
        self.res = res
        L.moe_block_pre_norm_fwd(self.desc, res, self.params["pre_w"], self.params.get("pre_b"),
                                 self.x, stream)
        return self.x

    def forward(self, res, logits, bias=None, gate=None, stream=None, timer=None, mask=None,
                seq_offsets=None):
        """res [T,d] (kept for the backward) -> res_out; logits, bias, mask and
        seq_offsets: the router's, as MoEExpertMLP.forward; gate fp32 [T] with a
        token gate.  A router that reads x calls forward_norm first; the norm runs
        again here, with the same result."""
        if self.token_gate and gate is None:
            raise ValueError("a token gate needs its values")
        layer, t = self.layer, self.layer._t
        layer._check_loss_inputs(mask, seq_offsets)
        self.gate = gate if self.token_gate else self.params.get("gate")
        with t(timer, "pre_norm"):
            self.forward_norm(res, stream)
        layer.route(self.x, logits, bias, stream, timer, mask, seq_offsets)
        layer.mlp_forward(stream, timer)
        with t(timer, "combine_post_norm"):
            L.moe_block_post_norm_fwd(
                self.desc, res, layer.y, dict(self.params, gate=self.gate), self.res_out, None,
                dict(row_of=layer.row_of, topk_w=layer.topk_w, y_out=layer.out), stream)
        return self.res_out

    def backward_branch(self, dres_out, stream=None, timer=None, dloss=None):
        """Gradient of res_out back to the layer's input: layer.dx, layer.dlogits
        and the gradients of the post norm, gate and experts; dloss: as
        MoEExpertMLP.backward."""
        layer = self.layer
        with layer._t(timer, "post_norm_bwd"):
            L.moe_block_post_norm_bwd(self.desc, dres_out, None, None, layer.out,
                                      dict(self.params, gate=self.gate), None, self.dout,
                                      self.grads, self.ws, 1.0, stream)
        layer.backward(self.dout, stream, timer, dloss)
        return layer.dx

    def backward(self, dres_out, stream=None, timer=None, dloss=None):
        """dres_out [T,d] -> dres, the gradient of res through the residual, the
        norms and the experts.  The router's logits are an input, so their
        gradient (layer.dlogits) is not carried into x: a caller that made them
        from x calls backward_branch, adds its part to layer.dx and calls
        backward_norm."""
        self.backward_branch(dres_out, stream, timer, dloss)
        return self.backward_norm(dres_out, stream, timer)

    def backward_norm(self, dres_out, stream=None, timer=None):
        """dres = res_scale*dres_out + N1^T(layer.dx)."""
        with self.layer._t(timer, "pre_norm_bwd"):
            L.moe_block_pre_norm_bwd(self.desc, self.layer.dx, self.res, self.params["pre_w"],
                                     dres_out, self.dres, self.grads["pre_w"],
                                     self.grads.get("pre_b"), self.ws, self.res_scale, stream)
        return self.dres

    def clip_gradients(self, max_norm, eps=1e-6, norm_type="l2", stream=None):
        """Global norm of the block's gradients (self.norm, self.norms on the
        device, no host sync) and the gradients clipped in place."""
        L.moe_grad_norm(self.gradients, self.norm, self.norms, norm_type, self.norm_ws, stream)
        L.moe_clip_grads(self.gradients, self.norm, max_norm, eps, stream)
        return self.norm

    def step(self, res, logits, bias, dres_out, max_norm=None, gate=None, stream=None, timer=None,
             mask=None, seq_offsets=None, dloss=None):
        """One forward and backward of the block, gradients clipped, and where
        orthogonal_updates() asked for them the experts' updates."""
        self.forward(res, logits, bias, gate, stream, timer, mask, seq_offsets)
        self.backward(dres_out, stream, timer, dloss)
        if max_norm is not None:
            self.clip_gradients(max_norm, stream=stream)
        if self.updates is not None:
            with self.layer._t(timer, "updates"):
                self.updates.step(stream)
        return self.dres
