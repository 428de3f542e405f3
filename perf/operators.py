"""Measured cases of the residual-block norms and of gradient clipping.

What a residual block around the routed-expert MLP needs besides the MLP:

* the norm before it (``pre``): x = N1(r), and its gradient joined to the
  residual's, dr = s dr' + N1^T(dx);
* the norm, gate and scaled residual after it (``post``):
  r' = a r + b G * N2(y), where wanted with the next block's norm
  x' = N1(r') in the same pass, and on a routed layer with y combined from the
  expert rows, y[t] = sum_s w[t,s] Y[row_of[t,s]]; and its gradient;
* the global norm of a list of gradients and their clipped copies,
  out = g * min(1, max_norm / (norm + 1e-6)).

N is an RMS norm, xhat = v / sqrt(mean(v^2) + eps), or a layer norm,
xhat = (v - mean) / sqrt(var + eps), followed by xhat * (offset + w) + c.
The gate G is a vector over the channels, a number for each token or a full
tensor, used as it is or through a sigmoid or tanh.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_CLIP_EPS = 1e-6


# ------------------------------------------------------------------ cases
def _norm(op, T, d, pre="rms", post=None, gate=None, gate_act="none", act="bf16", res="bf16",
          par="bf16", bias=False, offset=0.0, a=1.0, b=1.0, k=0, pitched=False):
    return dict(op=op, T=T, d=d, pre=pre, post=post, gate=gate, gate_act=gate_act, act=act,
                res=res, par=par, bias=bias, offset=offset, a=a, b=b, k=k, pitched=pitched)


def _grads(layers, E, d, F, dtype="bf16", out="bf16", max_norm=1.0, kind="l2"):
    return dict(op="clip", layers=layers, E=E, d=d, F=F, dtype=dtype, out=out, max_norm=max_norm,
                kind=kind)


def listed():
    return [
        # one token being decoded, at the clamped-SwiGLU layer's width
        dict(_norm("pre_fwd", 1, 2880), name="pre_fwd_one_token"),
        # the default training batch of the 64-expert layer, layer norm with bias
        dict(_norm("pre_fwd", 4096, 2048, pre="layer", bias=True), name="pre_fwd_layer_t4096"),
        # the dense sweep's 16384 rows, weights stored around zero
        dict(_norm("pre_bwd", 16384, 4096, offset=1.0), name="pre_bwd_t16384_d4096"),
        # eight sequences decoded together: norm, channel gate, next block's norm
        dict(_norm("post_fwd", 8, 7168, post="rms", gate="channel"), name="post_fwd_decode_t8"),
        # a long prompt with the residual stream kept in 32 bits
        dict(_norm("post_fwd", 16384, 7168, post="rms", gate="channel", res="fp32", par="fp32",
                   a=0.75, b=0.5), name="post_fwd_t16384_res32"),
        # a routed layer's expert rows combined, normed and added, k = 4
        dict(_norm("routed_fwd", 16384, 2880, post="rms", k=4), name="routed_fwd_t16384_k4"),
        # odd width and token count, 32-bit tensors, gate tensor, views of wider buffers
        dict(_norm("post_bwd", 1001, 1441, pre="layer", post="layer", gate="full",
                   gate_act="tanh", act="fp32", res="fp32", par="fp32", bias=True,
                   pitched=True), name="post_bwd_odd_full_gate"),
        # the 64-expert layer's batch, a sigmoid gate for each token, no next norm
        dict(_norm("post_bwd", 4096, 2048, pre=None, post="rms", gate="token",
                   gate_act="sigmoid"), name="post_bwd_token_gate_t4096"),
        # the widest layer's training batch: both norms' gradients in one pass
        dict(_norm("post_bwd", 16384, 7168, post="rms", gate="channel", a=0.75, b=0.5),
             name="post_bwd_t16384_d7168"),
        # a small model: many small 32-bit tensors
        dict(_grads(12, 8, 256, 512, dtype="fp32", out="fp32"), name="clip_12_small_layers"),
        # the 64-expert layer's gradients into the optimizer's 32-bit buffers
        dict(_grads(1, 64, 2048, 1408, out="fp32"), name="clip_e64_d2048"),
        # the widest layer's 32 local experts, clipped in their own type
        dict(_grads(1, 32, 7168, 2048), name="clip_e32_d7168"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    while True:
        c = _draw_grads(rng) if rng.random() < 0.3 else _draw_norm(rng)
        if work(c)["bytes"] <= most and 3072 not in _sizes(c):
            return c


def _draw_grads(rng):
    E, d, F = _log_int(rng, 1, 64), 64 * _log_int(rng, 1, 112), 32 * _log_int(rng, 1, 64)
    one = math.prod(_shapes(_grads(1, E, d, F))[0])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    return _grads(_log_int(rng, 1, max(1, min(24, (1 << 29) // one))), E, d, F, dtype=dtype,
                  out="fp32" if dtype == "fp32" else rng.choice(["bf16", "fp32"]),
                  max_norm=rng.choice([0.5, 1.0, 1.0, 1e6]), kind=rng.choice(["l2", "l2", "l2", "inf"]))


def _draw_norm(rng):
    op = rng.choice(["pre_fwd", "pre_bwd", "post_fwd", "post_fwd", "routed_fwd", "post_bwd",
                     "post_bwd"])
    T = _log_int(rng, 1, 16384)
    d = _log_int(rng, 64, 7168) if rng.random() < 0.3 else 64 * _log_int(rng, 1, 112)
    act, res = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
    post = rng.choice(["rms", "rms", "layer"]) if op.startswith(("post", "routed")) else None
    gate = rng.choice([None, "channel", "channel", "token", "full"]) if post else None
    if gate and rng.random() < 0.15:
        post = None                       # a gated residual without a norm
    pre = rng.choice(["rms", "rms", "layer"])
    if not op.startswith("pre") and rng.random() < 0.3:
        pre = None                        # the last block: no norm follows
    return _norm(op, T, d, pre=pre, post=post, gate=gate,
                 gate_act=rng.choice(["none", "sigmoid", "tanh"]) if gate else "none", act=act,
                 res=res, par=rng.choice([act, "fp32"]), bias=rng.random() < 0.3,
                 offset=rng.choice([0.0, 1.0]), a=rng.choice([1.0, 0.75]),
                 b=rng.choice([1.0, 0.5]), k=rng.choice([1, 2, 4, 6, 8]) * (op == "routed_fwd"),
                 pitched=rng.random() < 0.3)


def _sizes(c):
    if c["op"] == "clip":
        return {c["E"], c["d"], c["F"]} | {n for shape in _shapes(c) for n in shape}
    return {c["T"], c["d"], c["d"] + 72, c["T"] * c["k"], _capacity(c)}


# ----------------------------------------------------------------- inputs
def _capacity(c):
    """Rows of the expert-row buffer: every (token, slot), rounded up to 128."""
    return (c["T"] * c["k"] + 127) // 128 * 128


def _eps(kind):
    return 1e-5 if kind == "layer" else 1e-6


def _shapes(c):
    """Gradient tensors of `layers` routed-expert layers: FC1 in its packed
    order, FC2, their biases, the router and the block's two norms."""
    Fp = (c["F"] + 127) // 128 * 128
    one = [(c["E"], 2 * Fp, c["d"]), (c["E"], c["d"], c["F"]), (c["E"], 2 * Fp),
           (c["E"], c["d"]), (c["E"], c["d"]), (c["d"],), (c["d"],)]
    return one * c["layers"]


def _inputs(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if c["op"] == "clip":
        tensors = []
        for i, shape in enumerate(_shapes(c)):
            t = torch.empty(shape, dtype=_TYPES[c["dtype"]], device="cuda")
            t.normal_(0.0, 10.0 ** -(2 + i % 3), generator=g)
            if len(shape) == 3 and shape[0] > 4:
                t[i % shape[0]].zero_()                       # an expert without tokens
            tensors.append(t)
        return dict(grads=tensors)

    T, d, act, res, par = c["T"], c["d"], _TYPES[c["act"]], _TYPES[c["res"]], _TYPES[c["par"]]

    def rows(n, dtype, scale):
        t = randn(n, d).mul_(scale)
        if dtype is not act or c["op"] in ("pre_fwd", "pre_bwd"):
            t[:, :: 97] *= 12.0                               # a residual's few large channels
        if not c["pitched"]:
            return t.to(dtype)
        wide = torch.zeros((n, d + 72), dtype=dtype, device="cuda")
        wide[:, 8:8 + d] = t
        return wide[:, 8:8 + d]

    s = {}
    for n, on in (("pre", c["pre"]), ("post", c["post"])):
        s[n + "_w"] = (1.0 - c["offset"] + 0.1 * randn(d)).to(par) if on else None
        s[n + "_b"] = (0.1 * randn(d)).to(par) if on and c["bias"] else None
    s["gate"] = None
    if c["gate"] == "channel":
        s["gate"] = (0.5 + 0.2 * randn(d)).to(par)
    elif c["gate"] == "token":
        s["gate"] = randn(T)
    elif c["gate"] == "full":
        s["gate"] = rows(T, act, 1.0)
    if c["op"] in ("pre_fwd", "post_fwd", "routed_fwd", "pre_bwd"):
        s["res"] = rows(T, res, 2.0)
    if c["op"] == "routed_fwd":
        k = c["k"]
        s["y"] = rows(_capacity(c), act, 0.7)
        perm = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32)
        s["row_of"] = perm.view(T, k)
        s["topk_w"] = torch.softmax(randn(T, k), dim=1)
    elif c["op"] in ("post_fwd", "post_bwd"):
        s["y"] = rows(T, act, 0.7)
    if c["op"] in ("pre_bwd", "post_bwd"):
        s["dres_in"] = rows(T, res, 1e-2)
        if c["pre"]:
            s["dx"] = rows(T, act, 1e-2)
            if c["op"] == "post_bwd":
                s["res_out"] = rows(T, res, 2.0)
    return s


def prepare(case, seed):
    c, s = case, _inputs(case, seed)
    s["case"] = c
    if c["op"] == "clip":
        # the optimizer's flat buffer, and its piece for each tensor
        sizes = [t.numel() for t in s["grads"]]
        s["flat"] = torch.empty(sum(sizes), dtype=_TYPES[c["out"]], device="cuda")
        s["outs"] = [f.view(t.shape) for f, t in zip(s["flat"].split(sizes), s["grads"])]
        if own:
            import moe_expert_mlp_gb300 as m
            s["list"] = m.GradList(s["grads"], s["outs"])
            s["ws"] = torch.empty(m.moe_grad_norm_workspace_size(len(s["grads"])),
                                  dtype=torch.uint8, device="cuda")
        return s
    if own:
        import moe_expert_mlp_gb300 as m
        s["desc"] = m.make_block_norm_desc(
            c["T"], c["d"], dtype=c["act"], res_dtype=c["res"], param_dtype=c["par"],
            pre_norm=c["pre"], post_norm=c["post"], pre_eps=_eps(c["pre"]),
            post_eps=_eps(c["post"]), pre_offset=c["offset"], post_offset=c["offset"],
            gate=c["gate"], gate_act=c["gate_act"], res_scale=c["a"], branch_scale=c["b"])
        s["ws"] = torch.empty(m.moe_block_norm_workspace_size(s["desc"]), dtype=torch.uint8,
                              device="cuda")
    return s


# ------------------------------------------------------------- plain forms
def _xhat(v, kind, eps):
    """Normalised rows and 1 / sqrt(. + eps), in 32 bits."""
    v = v.float()
    if kind == "layer":
        v = v - v.mean(dim=1, keepdim=True)
    rstd = torch.rsqrt((v * v).mean(dim=1, keepdim=True) + eps)
    return v * rstd, rstd


def _affine(xh, w, b, offset):
    out = xh * (w.float() + offset)
    return out if b is None else out + b.float()


def _norm_grad(dn, xh, rstd, w, kind, offset):
    """Gradients of n = xh * (offset + w) + c by its input, w and c."""
    dxh = dn * (w.float() + offset)
    dv = dxh - xh * (dxh * xh).mean(dim=1, keepdim=True)
    if kind == "layer":
        dv = dv - dxh.mean(dim=1, keepdim=True)
    return dv * rstd, (dn * xh).sum(dim=0), dn.sum(dim=0)


def _gate(s):
    """Gate value and the derivative of its activation, shaped to broadcast."""
    c, g = s["case"], s["gate"]
    if g is None:
        return 1.0, None
    g = g.float()
    if c["gate"] == "token":
        g = g[:, None]
    if c["gate_act"] == "sigmoid":
        v = torch.sigmoid(g)
        return v, v * (1 - v)
    if c["gate_act"] == "tanh":
        v = torch.tanh(g)
        return v, 1 - v * v
    return g, torch.ones_like(g)


def _plain_fwd(s):
    c = s["case"]
    act, res = _TYPES[c["act"]], _TYPES[c["res"]]
    if c["op"] == "pre_fwd":
        xh, _ = _xhat(s["res"], c["pre"], _eps(c["pre"]))
        return {"x": _affine(xh, s["pre_w"], s["pre_b"], c["offset"]).to(act)}
    out = {}
    y = s["y"]
    if c["op"] == "routed_fwd":
        picked = y[s["row_of"].long().view(-1)].float().view(c["T"], c["k"], c["d"])
        y = (picked * s["topk_w"][:, :, None]).sum(dim=1)
        out["y"] = y.to(act)
    n = y.float()
    if c["post"]:
        n = _affine(_xhat(y, c["post"], _eps(c["post"]))[0], s["post_w"], s["post_b"], c["offset"])
    r = c["a"] * s["res"].float() + c["b"] * _gate(s)[0] * n
    out["res"] = r.to(res)
    if c["pre"]:
        xh, _ = _xhat(r, c["pre"], _eps(c["pre"]))
        out["x"] = _affine(xh, s["pre_w"], s["pre_b"], c["offset"]).to(act)
    return out


def _plain_bwd(s):
    c = s["case"]
    act, res, par = _TYPES[c["act"]], _TYPES[c["res"]], _TYPES[c["par"]]
    out = {}
    dr = c["a"] * s["dres_in"].float()
    if c["pre"]:
        v = s["res"] if c["op"] == "pre_bwd" else s["res_out"]
        xh, rstd = _xhat(v, c["pre"], _eps(c["pre"]))
        dv, dw, db = _norm_grad(s["dx"].float(), xh, rstd, s["pre_w"], c["pre"], c["offset"])
        dr = dr + dv
        out["dpre_w"] = dw.to(par)
        if c["bias"]:
            out["dpre_b"] = db.to(par)
        out["dres"] = dr.to(res)
    if c["op"] == "pre_bwd":
        return out
    n = y = s["y"].float()
    if c["post"]:
        xh, rstd = _xhat(y, c["post"], _eps(c["post"]))
        n = _affine(xh, s["post_w"], s["post_b"], c["offset"])
    G, dG = _gate(s)
    if c["gate"]:
        dg = c["b"] * dr * n * dG
        if c["gate"] == "channel":
            out["dgate"] = dg.sum(dim=0).to(par)
        elif c["gate"] == "token":
            out["dgate"] = dg.sum(dim=1)
        else:
            out["dgate"] = dg.to(act)
    dn = c["b"] * G * dr
    if c["post"]:
        dn, dw, db = _norm_grad(dn, xh, rstd, s["post_w"], c["post"], c["offset"])
        out["dpost_w"] = dw.to(par)
        if c["bias"]:
            out["dpost_b"] = db.to(par)
    out["dy"] = dn.to(act)
    return out


def _plain_grads(s):
    c = s["case"]
    if c["kind"] == "inf":
        norms = torch.stack([t.abs().max().float() for t in s["grads"]])
        total = norms.max()
    else:
        squares = torch.stack([t.float().square().sum() for t in s["grads"]])
        norms, total = squares.sqrt(), squares.sum().sqrt()
    scale = torch.clamp(c["max_norm"] / (total + _CLIP_EPS), max=1.0)
    for t, o in zip(s["grads"], s["outs"]):
        o.copy_(t.float() * scale)
    return {"norm": total.view(1), "norms": norms, "grads": s["flat"]}


# --------------------------------------------------- the framework's calls
def _own_fwd(s):
    import moe_expert_mlp_gb300 as m
    c, T, d = s["case"], s["case"]["T"], s["case"]["d"]
    act, res = _TYPES[c["act"]], _TYPES[c["res"]]
    x = torch.empty((T, d), dtype=act, device="cuda") if c["pre"] else None
    if c["op"] == "pre_fwd":
        m.moe_block_pre_norm_fwd(s["desc"], s["res"], s["pre_w"], s["pre_b"], x)
        return {"x": x}
    out = {}
    r = torch.empty((T, d), dtype=res, device="cuda")
    routed = None
    if c["op"] == "routed_fwd":
        out["y"] = torch.empty((T, d), dtype=act, device="cuda")
        routed = dict(row_of=s["row_of"], topk_w=s["topk_w"], y_out=out["y"])
    m.moe_block_post_norm_fwd(s["desc"], s["res"], s["y"], s, r, x, routed)
    out["res"] = r
    if c["pre"]:
        out["x"] = x
    return out


def _own_bwd(s):
    import moe_expert_mlp_gb300 as m
    c, T, d = s["case"], s["case"]["T"], s["case"]["d"]
    act, res, par = _TYPES[c["act"]], _TYPES[c["res"]], _TYPES[c["par"]]
    grads, out = {}, {}
    for n in ("pre", "post"):
        if c[n]:
            grads[n + "_w"] = out["d%s_w" % n] = torch.empty(d, dtype=par, device="cuda")
            if c["bias"]:
                grads[n + "_b"] = out["d%s_b" % n] = torch.empty(d, dtype=par, device="cuda")
    dres = torch.empty((T, d), dtype=res, device="cuda") if c["pre"] else None
    if c["pre"]:
        out["dres"] = dres
    if c["op"] == "pre_bwd":
        m.moe_block_pre_norm_bwd(s["desc"], s["dx"], s["res"], s["pre_w"], s["dres_in"], dres,
                                 grads["pre_w"], grads.get("pre_b"), s["ws"], c["a"])
        return out
    if c["gate"]:
        shape, dtype = {"channel": ((d,), par), "token": ((T,), torch.float32),
                        "full": ((T, d), act)}[c["gate"]]
        grads["gate"] = out["dgate"] = torch.empty(shape, dtype=dtype, device="cuda")
    out["dy"] = torch.empty((T, d), dtype=act, device="cuda")
    m.moe_block_post_norm_bwd(s["desc"], s["dres_in"], s.get("dx"), s.get("res_out"), s["y"], s,
                              dres, out["dy"], grads, s["ws"], c["a"])
    return out


def _own_grads(s):
    import moe_expert_mlp_gb300 as m
    c = s["case"]
    norm = torch.empty(1, dtype=torch.float32, device="cuda")
    norms = torch.empty(len(s["grads"]), dtype=torch.float32, device="cuda")
    m.moe_grad_norm(s["list"], norm, norms, c["kind"], s["ws"])
    m.moe_clip_grads(s["list"], norm, c["max_norm"], _CLIP_EPS)
    return {"norm": norm, "norms": norms, "grads": s["flat"]}


def run(state):
    op = state["case"]["op"]
    if op == "clip":
        out = _own_grads(state) if own else _plain_grads(state)
    elif op.endswith("fwd"):
        out = _own_fwd(state) if own else _plain_fwd(state)
    else:
        out = _own_bwd(state) if own else _plain_bwd(state)
    return {n: out[n] for n in sorted(out)}


# ------------------------------------------------------------------- work
def work(case):
    c = case
    size = {"bf16": 2, "fp32": 4}
    if c["op"] == "clip":
        n = sum(math.prod(s) for s in _shapes(c))
        return {"bytes": n * (size[c["dtype"]] + size[c["out"]]), "flops": 3 * n}
    n, a, r, p = c["T"] * c["d"], size[c["act"]], size[c["res"]], size[c["par"]] * c["d"]
    params = p * (bool(c["pre"]) + bool(c["post"])) * (2 if c["bias"] else 1)
    gate = {None: 0, "channel": p, "token": 4 * c["T"], "full": n * a}[c["gate"]]
    if c["op"] == "pre_fwd":
        return {"bytes": n * (r + a) + params, "flops": 5 * n}
    if c["op"] == "pre_bwd":
        return {"bytes": n * (3 * r + a) + 2 * params, "flops": 14 * n}
    pre = bool(c["pre"])
    if c["op"] == "post_bwd":
        return {"bytes": n * (r + 2 * a + pre * (2 * r + a)) + 2 * params + 2 * gate,
                "flops": (16 + 12 * pre) * n}
    k = c["k"] if c["op"] == "routed_fwd" else 0
    y = (k + 1) * n * a + 8 * k * c["T"] if k else n * a
    return {"bytes": n * (2 * r + pre * a) + y + params + gate,
            "flops": (9 + 5 * pre + 2 * k) * n}


# ------------------------------------------------------------------ exact
def _norm64(v, kind, w, b, offset):
    if kind is None:
        return v
    m = v.mean(-1, keepdim=True) if kind == "layer" else 0.0
    q = (v - m) / ((v - m).pow(2).mean(-1, keepdim=True) + _eps(kind)).sqrt()
    q = q * (offset + w)
    return q + b if b is not None else q


def _branch64(c, y, s):
    n = _norm64(y, c["post"], s["post_w"], s["post_b"], c["offset"])
    g = s["gate"]
    if g is None:
        return c["b"] * n
    g = {"none": lambda v: v, "sigmoid": lambda v: 1 / (1 + (-v).exp()),
         "tanh": lambda v: 1 - 2 / ((2 * v).exp() + 1)}[c["gate_act"]](g)
    return c["b"] * n * (g.unsqueeze(-1) if c["gate"] == "token" else g)


def exact(case, seed):
    c, raw = case, _inputs(case, seed)
    if c["op"] == "clip":
        return _exact_grads(c, raw["grads"])
    s = {n: (t.double() if t is not None and t.is_floating_point() else t) for n, t in raw.items()}
    if c["op"] == "pre_fwd":
        return {"x": _norm64(s["res"], c["pre"], s["pre_w"], s["pre_b"], c["offset"])}
    out = {}
    if c["op"].endswith("fwd"):
        y = s["y"]
        if c["op"] == "routed_fwd":
            y = sum(s["topk_w"][:, i, None] * s["y"][s["row_of"][:, i].long()]
                    for i in range(c["k"]))
            out["y"] = y
        out["res"] = c["a"] * s["res"] + _branch64(c, y, s)
        if c["pre"]:
            out["x"] = _norm64(out["res"], c["pre"], s["pre_w"], s["pre_b"], c["offset"])
        return {n: out[n] for n in sorted(out)}
    # gradients by differentiating the 64-bit forward
    dr = c["a"] * s["dres_in"]
    if c["pre"]:
        leaves = {"dres": s["res" if c["op"] == "pre_bwd" else "res_out"], "dpre_w": s["pre_w"]}
        if c["bias"]:
            leaves["dpre_b"] = s["pre_b"]
        for t in leaves.values():
            t.requires_grad_()
        n = _norm64(leaves["dres"], c["pre"], s["pre_w"], s["pre_b"], c["offset"])
        out.update(zip(leaves, torch.autograd.grad(n, list(leaves.values()), s["dx"])))
        dr = out["dres"] = out["dres"] + dr
    if c["op"] == "post_bwd":
        leaves = {"dy": s["y"]}
        if c["post"]:
            leaves["dpost_w"] = s["post_w"]
            if c["bias"]:
                leaves["dpost_b"] = s["post_b"]
        if c["gate"]:
            leaves["dgate"] = s["gate"]
        for t in leaves.values():
            t.requires_grad_()
        out.update(zip(leaves, torch.autograd.grad(_branch64(c, s["y"], s), list(leaves.values()),
                                                   dr)))
    return {n: out[n] for n in sorted(out)}


def _exact_grads(c, grads):
    def pieces(t):
        flat = t.reshape(-1)
        return (flat[i:i + (1 << 27)].double() for i in range(0, flat.numel(), 1 << 27))

    if c["kind"] == "inf":
        norms = torch.stack([torch.stack([p.abs().amax() for p in pieces(t)]).amax()
                             for t in grads])
        total = norms.amax()
    else:
        norms = torch.stack([sum((p @ p for p in pieces(t)), torch.zeros((), device="cuda").double())
                             for t in grads]).sqrt()
        total = torch.linalg.vector_norm(norms)
    scale = min(1.0, c["max_norm"] / (float(total) + _CLIP_EPS))
    flat = torch.cat([p for t in grads for p in pieces(t)]).mul_(scale)
    return {"grads": flat, "norm": total.view(1), "norms": norms}
