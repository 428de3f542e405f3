"""Measured cases of a routed layer's training step beside its products: the
router's losses with their gradient, and orthogonalised weight updates.

* the router's losses (``loss_fwd``): with p = softmax(logits) over the experts,
  for each sequence s of tokens its per-expert counts c[s,e], f = E c / (k N_s)
  and P[s,e] = mean_t p[t,e],
      balance = sum_s (N_s / N) sum_e f[s,e] P[s,e]
      z       = (1/N) sum_t logsumexp(logits[t])^2
      loss    = balance_coef * balance + z_coef * z;
* their gradient (``loss_bwd``), f held fixed, joined to the gradient that the
  selected experts' weights give,
      dlogits[t,e] = dloss / N * p (balance_coef (f - sum_j f_j p_j)
                                    + 2 z_coef logsumexp)
                     + [e = idx[t,i]] w_i (dw_i - sum_j w_j dw_j);
* orthogonalised updates (``ortho``): a momentum m' = momentum*m +
  (1 - dampening)*g, U = m' or (Nesterov) (1 - dampening)*g + momentum*m', then
  for each matrix X = U / (|U|_F + eps) and `steps` times
      A = X X^T,  X <- a X + (b A + c A^2) X,
  times a scale (X^T X on the other side gives the same for tall matrices).
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_EPS = 1e-7


# ------------------------------------------------------------------ cases
def _loss(op, T, E, k, seqs=0, masked=False, routed=False, balance=1e-2, z=1e-3, off=False):
    return dict(op=op, T=T, E=E, k=k, seqs=seqs, masked=masked, routed=routed, balance=balance,
                z=z, off=off)


def _ortho(batch, rows, cols, grad="bf16", momentum=0.0, nesterov=False, dampening=0.0, steps=5,
           scale=1.0, pitched=False):
    return dict(op="ortho", batch=batch, rows=rows, cols=cols, grad=grad, momentum=momentum,
                nesterov=nesterov, dampening=dampening, steps=steps, scale=scale, pitched=pitched)


def listed():
    return [
        # the small model's batch: what a call costs
        dict(_loss("loss_fwd", 256, 8, 2), name="loss_fwd_t256_e8"),
        # the 64-expert layer's batch, one balance over all its tokens
        dict(_loss("loss_fwd", 4096, 64, 6), name="loss_fwd_t4096_e64"),
        # a long-context batch: 16 packed sequences, padding, rows past the last
        dict(_loss("loss_fwd", 65536, 256, 8, seqs=16, masked=True), name="loss_fwd_t65536_e256"),
        # the 64-expert layer's whole router gradient
        dict(_loss("loss_bwd", 4096, 64, 6, routed=True), name="loss_bwd_t4096_e64"),
        # odd sizes, an expert switched off, padding, no gradient of the weights
        dict(_loss("loss_bwd", 1001, 61, 4, seqs=3, masked=True, off=True),
             name="loss_bwd_odd_t1001_e61"),
        # the long-context batch's whole router gradient
        dict(_loss("loss_bwd", 65536, 256, 8, seqs=16, masked=True, routed=True),
             name="loss_bwd_t65536_e256"),
        # the 64-expert layer's router weight: one flat matrix, kept in 32 bits
        dict(_ortho(1, 64, 2048, grad="fp32", momentum=0.95, nesterov=True), name="ortho_router"),
        # the small model's experts
        dict(_ortho(8, 256, 512), name="ortho_8_small"),
        # odd sizes, 32-bit gradients, views of wider buffers, plain momentum
        dict(_ortho(3, 1001, 1441, grad="fp32", momentum=0.9, dampening=0.1, scale=0.2 * 37.96,
                    pitched=True), name="ortho_odd"),
        # clamped-SwiGLU layer, a few local experts' FC2: square matrices
        dict(_ortho(4, 2880, 2880, momentum=0.95, nesterov=True, dampening=0.05),
             name="ortho_4_square"),
        # the 64-expert layer's FC2, tall matrices
        dict(_ortho(64, 2048, 1408, momentum=0.95, nesterov=True, dampening=0.05),
             name="ortho_64_tall"),
        # the widest layer's 32 local experts, FC2
        dict(_ortho(32, 7168, 2048, momentum=0.95, nesterov=True, dampening=0.05, scale=1.87),
             name="ortho_32_widest"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(c):
    """Operations of the plain products, and elements."""
    m, n = sorted((c["rows"], c["cols"]))
    return c["batch"] * c["steps"] * (4 * m * m * n + 2 * m ** 3), c["batch"] * m * n


def draw(rng):
    most = listed()[-1]
    while True:
        if rng.random() < 0.5:
            E = _log_int(rng, 4, 256)
            c = _loss(rng.choice(["loss_fwd", "loss_bwd"]), _log_int(rng, 64, 65536), E,
                      rng.randint(1, min(8, E // 2)), seqs=rng.choice([0, 0, 1, 4, 32]),
                      masked=rng.random() < 0.4, routed=rng.random() < 0.6,
                      balance=rng.choice([1e-2, 1e-3]), z=rng.choice([0.0, 1e-3]),
                      off=rng.random() < 0.2)
            if c["op"] == "loss_fwd":
                c["routed"] = False
            return c
        momentum = rng.choice([0.0, 0.9, 0.95])
        c = _ortho(_log_int(rng, 1, 64), _log_int(rng, 64, 7168), _log_int(rng, 64, 7168),
                   grad=rng.choice(["bf16", "bf16", "fp32"]), momentum=momentum,
                   nesterov=momentum > 0 and rng.random() < 0.5,
                   dampening=rng.choice([0.0, 0.05]) if momentum else 0.0,
                   steps=rng.choice([3, 5, 5]), scale=rng.choice([1.0, 0.2]),
                   pitched=rng.random() < 0.3)
        if rng.random() < 0.6:
            c["rows"], c["cols"] = (max(64, v // 64 * 64) for v in (c["rows"], c["cols"]))
        if all(x <= y for x, y in zip(_cost(c), _cost(most))):
            return c


# ----------------------------------------------------------------- inputs
def _inputs(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if c["op"] == "ortho":
        return _matrices(c, g, randn)
    T, E, k, S = c["T"], c["E"], c["k"], max(c["seqs"], 1)
    s = {}
    # a trained router: some experts liked more, confident tokens
    s["logits"] = 1.5 * randn(T, E) + 0.7 * randn(E)
    if c["off"]:
        s["logits"][:, E // 2] = -math.inf
    top = torch.topk(s["logits"], k, dim=1)
    s["topk_idx"] = top.indices.to(torch.int32)
    s["topk_w"] = torch.softmax(top.values, dim=1)
    s["mask"] = torch.rand(T, generator=g, device="cuda") > 0.1 if c["masked"] else None
    s["offsets"] = None
    if c["seqs"]:
        # ragged sequences, one of them empty where there are several, and a
        # few rows of padding behind the last
        cuts = torch.rand(S - 1, generator=g, device="cuda").sort().values
        offsets = torch.zeros(S + 1, device="cuda")
        offsets[1:S] = (cuts * (T - T // 16)).floor()
        offsets[S] = T - T // 16
        if S > 2:
            offsets[2] = offsets[1]
        s["offsets"] = offsets.to(torch.int32)
    if c["op"] == "loss_bwd":
        seg, live = _segments(c, s)
        live = live.to(torch.int32)
        s["tokens"] = torch.zeros(S + 1, dtype=torch.int32, device="cuda")
        s["tokens"][:S].index_add_(0, seg, live)
        s["tokens"][S:] = live.sum()
        s["counts"] = _counts(c, s, seg, live)
        s["dloss"] = torch.full((1,), 1.0, device="cuda")
        if c["routed"]:
            s["dw"] = randn(T, k) * (0.1 / T)
    return s


def _matrices(c, g, randn):
    """Gradients as a step makes them: products over an expert's few or many
    tokens, none for some experts; a momentum of other steps' gradients."""
    B, R, C = c["batch"], c["rows"], c["cols"]

    def stack(dtype):
        if not c["pitched"]:
            return torch.zeros((B, R, C), dtype=dtype, device="cuda")
        wide = torch.zeros((B, R + 3, C + 24), dtype=dtype, device="cuda")
        return wide[:, 1:1 + R, 8:8 + C]

    s = {"grad": stack(_TYPES[c["grad"]]), "mom": stack(torch.float32) if c["momentum"] else None}
    for i in range(B):
        tokens = (min(R, C), 512, 24, 2 * max(R, C))[i % 4]
        if i % 16 != 5:                                       # else an expert without tokens
            t = randn(R, tokens) @ randn(tokens, C)
            s["grad"][i] = t.mul_(1e-3 / math.sqrt(tokens))
        if c["momentum"]:
            s["mom"][i] = randn(R, C).mul_(2e-4)
    return s


def prepare(case, seed):
    c, s = case, _inputs(case, seed)
    s["case"] = c
    if own:
        import moe_expert_mlp_gb300 as m
        if c["op"] == "ortho":
            s["desc"] = m.make_orthogonalize_desc(
                c["batch"], c["rows"], c["cols"], grad_dtype=c["grad"], steps=c["steps"], eps=_EPS,
                momentum=c["momentum"], dampening=c["dampening"], nesterov=c["nesterov"],
                scale=c["scale"])
            size = m.moe_orthogonalize_workspace_size(s["desc"])
        else:
            s["desc"] = m.make_router_loss_desc(c["T"], c["E"], c["k"], sequences=max(c["seqs"], 1),
                                                balance_coef=c["balance"], z_coef=c["z"])
            size = m.moe_router_loss_workspace_size(s["desc"])
        s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------- plain forms
def _segments(c, s):
    """Each token's sequence, and whether it counts."""
    t = torch.arange(c["T"], device="cuda")
    live = torch.ones(c["T"], dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
    if s["offsets"] is None:
        return torch.zeros_like(t), live
    S = c["seqs"]
    seg = torch.bucketize(t, s["offsets"][1:].long(), right=True)
    live = live & (seg < S) & (t >= s["offsets"][0])
    return seg.clamp(max=S - 1), live


def _counts(c, s, seg, live):
    S = max(c["seqs"], 1)
    at = seg[:, None] * c["E"] + s["topk_idx"].long()
    counts = torch.zeros(S * c["E"], dtype=torch.int32, device="cuda")
    counts.index_add_(0, at.view(-1), live.to(torch.int32)[:, None].expand(-1, c["k"]).reshape(-1))
    return counts.view(S, c["E"])


def _softmax(logits):
    top = logits.max(dim=1, keepdim=True).values
    e = torch.exp(logits - top)
    total = e.sum(dim=1, keepdim=True)
    return e / total, top + torch.log(total)


def _plain_loss(s):
    c = s["case"]
    S = max(c["seqs"], 1)
    p, lse = _softmax(s["logits"])
    seg, live = _segments(c, s)
    w = live.float()
    member = (seg[:, None] == torch.arange(S, device="cuda")) * w[:, None]     # [T, S]
    tokens = torch.zeros(S + 1, dtype=torch.int32, device="cuda")
    tokens[:S] = member.sum(dim=0).to(torch.int32)
    tokens[S] = tokens[:S].sum()
    counts = _counts(c, s, seg, live)
    per_seq = tokens[:S, None].float()
    probs = (member.t() @ p) / per_seq.clamp(min=1)
    f = counts.float() * (c["E"] / c["k"]) / per_seq.clamp(min=1)
    total = tokens[S].float().clamp(min=1)
    balance = (per_seq * f * probs).sum() / total
    z = (w * lse[:, 0] * lse[:, 0]).sum() / total
    loss = torch.stack([c["balance"] * balance + c["z"] * z, balance, z])
    return {"counts": counts, "loss": loss, "probs": probs, "tokens": tokens}


def _plain_loss_grad(s):
    c = s["case"]
    S = max(c["seqs"], 1)
    p, lse = _softmax(s["logits"])
    seg, live = _segments(c, s)
    per_seq = s["tokens"][:S, None].float().clamp(min=1)
    f = s["counts"].float() * (c["E"] / c["k"]) / per_seq - 1.0     # a constant changes nothing
    ft = f[seg]
    grad = p * (c["balance"] * (ft - (ft * p).sum(dim=1, keepdim=True)) + 2 * c["z"] * lse)
    grad = grad * (live.float()[:, None] * s["dloss"] / s["tokens"][S].float().clamp(min=1))
    if c["routed"]:
        w, dw = s["topk_w"], s["dw"]
        grad = grad.scatter_add(1, s["topk_idx"].long(),
                                w * (dw - (w * dw).sum(dim=1, keepdim=True)))
    return {"dlogits": grad}


def _update(c, g, m):
    """The momentum and the direction it gives."""
    if not c["momentum"]:
        return None, g
    m = c["momentum"] * m + (1 - c["dampening"]) * g
    return m, (1 - c["dampening"]) * g + c["momentum"] * m if c["nesterov"] else m


def _plain_ortho(s):
    c = s["case"]
    mom, x = _update(c, s["grad"].float(), None if s["mom"] is None else s["mom"])
    x = x / (torch.sqrt((x * x).sum(dim=(1, 2), keepdim=True)) + _EPS)
    tall = c["rows"] > c["cols"]
    x = x.transpose(1, 2) if tall else x
    for _ in range(c["steps"]):
        A = x @ x.transpose(1, 2)
        x = 3.4445 * x + (-4.7750 * A + 2.0315 * (A @ A)) @ x
    x = (x.transpose(1, 2) if tall else x) * c["scale"]
    out = {"out": x.to(torch.bfloat16).contiguous()}
    if mom is not None:
        out["mom"] = mom
    return out


# --------------------------------------------------- the framework's calls
def _own_loss(s):
    import moe_expert_mlp_gb300 as m
    c = s["case"]
    S = max(c["seqs"], 1)
    counts = torch.empty((S, c["E"]), dtype=torch.int32, device="cuda")
    probs = torch.empty((S, c["E"]), dtype=torch.float32, device="cuda")
    tokens = torch.empty(S + 1, dtype=torch.int32, device="cuda")
    loss = torch.empty(3, dtype=torch.float32, device="cuda")
    m.moe_router_loss_fwd(s["desc"], s["logits"], s["topk_idx"], s["mask"], s["offsets"], counts,
                          tokens, probs, loss, s["ws"])
    return {"counts": counts, "loss": loss, "probs": probs, "tokens": tokens}


def _own_loss_grad(s):
    import moe_expert_mlp_gb300 as m
    c = s["case"]
    dlogits = torch.empty((c["T"], c["E"]), dtype=torch.float32, device="cuda")
    routed = dict(dw=s["dw"], topk_w=s["topk_w"], topk_idx=s["topk_idx"]) if c["routed"] else None
    m.moe_router_loss_bwd(s["desc"], s["logits"], s["mask"], s["offsets"], s["counts"], s["tokens"],
                          s["dloss"], routed, dlogits)
    return {"dlogits": dlogits}


def _own_ortho(s):
    import moe_expert_mlp_gb300 as m
    c = s["case"]
    shape = (c["batch"], c["rows"], c["cols"])
    out = {"out": torch.empty(shape, dtype=torch.bfloat16, device="cuda")}
    if c["momentum"]:
        out["mom"] = torch.empty(shape, dtype=torch.float32, device="cuda")
    m.moe_orthogonalize(s["desc"], s["grad"], out["out"], s["ws"], s["mom"], out.get("mom"))
    return out


def run(state):
    op = state["case"]["op"]
    if op == "loss_fwd":
        return _own_loss(state) if own else _plain_loss(state)
    if op == "loss_bwd":
        return _own_loss_grad(state) if own else _plain_loss_grad(state)
    return _own_ortho(state) if own else _plain_ortho(state)


# ------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "ortho":
        m, n = sorted((c["rows"], c["cols"]))
        e = c["batch"] * m * n
        size = {"bf16": 2, "fp32": 4}[c["grad"]] + 2 + (8 if c["momentum"] else 0)
        # half of each symmetric product: X X^T and A A
        return {"bytes": e * size, "flops": c["batch"] * c["steps"] * (3 * m * m * n + m ** 3)}
    T, E, k, S = c["T"], c["E"], c["k"], max(c["seqs"], 1)
    bytes_ = 4 * T * E + (T if c["masked"] else 0)
    if c["op"] == "loss_fwd":
        return {"bytes": bytes_ + 4 * T * k + 8 * S * E, "flops": 6 * T * E}
    return {"bytes": bytes_ + 4 * T * E + 4 * S * E + (12 * T * k if c["routed"] else 0),
            "flops": 10 * T * E}


# ------------------------------------------------------------------ exact
def exact(case, seed):
    c, s = case, _inputs(case, seed)
    if c["op"] == "ortho":
        return _exact_ortho(c, s)
    x = s["logits"].double()
    T, E, k, S = c["T"], c["E"], c["k"], max(c["seqs"], 1)
    t = torch.arange(T, device="cuda")
    ends = [0, T] if s["offsets"] is None else s["offsets"].tolist()
    live = torch.ones_like(t).double() if s["mask"] is None else s["mask"].double()
    inside = [live * ((t >= a) & (t < b)) for a, b in zip(ends, ends[1:])]
    N = max(float(sum(inside).sum()), 1.0)
    hot = torch.zeros(T, E, dtype=torch.float64, device="cuda")
    hot.scatter_(1, s["topk_idx"].long(), 1.0)
    counts = torch.stack([i @ hot for i in inside])
    if c["op"] == "loss_bwd":
        x.requires_grad_()
    lse = torch.logsumexp(x, dim=1)
    p = torch.exp(x - lse[:, None])
    n = torch.stack([i.sum() for i in inside]).clamp(min=1.0)
    probs = torch.stack([i @ p for i in inside]) / n[:, None]
    balance = sum(float(a) / N * (E / (k * float(a)) * f * q).sum()
                  for a, f, q in zip(n, counts, probs))
    z = (sum(inside) * lse * lse).sum() / N
    loss = c["balance"] * balance + c["z"] * z
    if c["op"] == "loss_fwd":
        return {"counts": None, "loss": torch.stack([loss, balance, z]), "probs": probs,
                "tokens": None}
    total = loss * float(s["dloss"])
    if c["routed"]:
        # the selected weights' share: <dw, softmax of the chosen logits>
        chosen = torch.softmax(torch.gather(x, 1, s["topk_idx"].long()), dim=1)
        total = total + (s["dw"].double() * chosen).sum()
    return {"dlogits": torch.autograd.grad(total, x)[0]}


def _exact_ortho(c, s):
    """By polynomials of the Gram matrix: X_k = Q_k X_0 with Q_k a polynomial of
    A_0 = X_0 X_0^T, A_k = Q_k A_0 Q_k."""
    a, b, k3 = 3.4445, -4.7750, 2.0315
    outs, moms = [], []
    for i in range(c["batch"]):
        mom, x = _update(c, s["grad"][i].double(),
                         None if s["mom"] is None else s["mom"][i].double())
        if mom is not None:
            moms.append(mom.float())
        x = x / (torch.linalg.matrix_norm(x) + _EPS)
        if c["rows"] > c["cols"]:
            x = x.t()
        A, Q = x @ x.t(), None
        for step in range(c["steps"]):
            M = k3 * (A @ A) + b * A
            M.diagonal().add_(a)
            Q = M if Q is None else M @ Q
            if step + 1 < c["steps"]:
                A = M @ A @ M
        x = (Q @ x) * c["scale"]
        outs.append((x.t() if c["rows"] > c["cols"] else x).float())
    out = {"out": torch.stack(outs)}
    if moms:
        out["mom"] = torch.stack(moms)
    return out
