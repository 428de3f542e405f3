"""The residual block's norms on the GPU against the fp64 oracle.

Bounds: a stored value is off by half a step of its type relative to its size
(bf16 2^-8, fp32 2^-24), plus what its fp32 arithmetic may be off: C * 2^-24
times the magnitude of the terms it is added up from (the oracle gives it).
A row's sum takes at most 32 additions in a thread, 5 + 4 across the group;
with the elementwise steps, the square root and division, C = 128 for what
one norm gives, 256 behind two, and T + 192 more for a sum over T tokens."""
import numpy as np
import pytest
import torch

import oracle.block_oracle as B

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def check(name, got, ref, mag, c):
    err = c * U * np.broadcast_to(mag, ref.shape)
    bound = HALF[got.dtype] * (np.abs(ref) + err) + err + 1e-40
    g = f64(got)
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    assert np.isfinite(g).all(), name
    over = np.abs(g - ref) - bound
    at = np.unravel_index(np.argmax(over), over.shape) if over.size else None
    assert not over.size or over[at] <= 0, (name, at, g[at], ref[at], bound[at])


class Case:
    """Inputs of one shape and option set, on the GPU and as the oracle sees them."""

    def __init__(self, T, d, pre="rms", post="rms", gate=None, act=None, types="bf16/bf16/bf16",
                 bias=False, offset=0.0, a=0.75, b=0.5, pitch=0, shift=0, weights=True, seed=0):
        import moe_expert_mlp_gb300 as m
        self.m, self.T, self.d, self.gate_kind, self.act = m, T, d, gate, act
        names = types.split("/")
        self.at, self.rt, self.pt = (TYPES[n] for n in names)
        self.a, self.b, self.pitch, self.shift = a, b, pitch, shift
        self.pre, self.post = B.NormSpec(pre, 1e-5, offset), B.NormSpec(post, 1e-6, offset)
        self.desc = m.make_block_norm_desc(
            T, d, *names, pre_norm=pre, post_norm=post, pre_eps=1e-5, post_eps=1e-6,
            pre_offset=offset, post_offset=offset, gate=gate, gate_act=act, res_scale=a,
            branch_scale=b)
        self.g = torch.Generator().manual_seed(seed + 131 * T + d)
        self.ws = torch.empty(m.moe_block_norm_workspace_size(self.desc), dtype=torch.uint8,
                              device="cuda")
        self.p = {}
        for n, kind in (("pre", pre), ("post", post)):
            on = kind is not None and weights
            self.p[n + "_w"] = self.vector(1.0 - offset) if on else None
            self.p[n + "_b"] = self.vector(0.0) if kind is not None and bias else None
        self.p["gate"] = None
        if gate == "channel":
            self.p["gate"] = self.vector(0.5)
        elif gate == "token":
            self.p["gate"] = self.randn(T).cuda()
        elif gate == "full":
            self.p["gate"] = self.rows(self.at)
        self.q = {n: f64(t) for n, t in self.p.items()}

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.g)

    def vector(self, mid):
        v = (mid + 0.3 * self.randn(self.d)).to(self.pt)
        wide = torch.zeros(self.d + self.shift, dtype=self.pt, device="cuda")
        wide[self.shift:] = v
        return wide[self.shift:]

    def empty(self, dtype, fill=None):
        wide = torch.full((self.T, self.d + self.pitch), float("nan"), dtype=dtype, device="cuda")
        v = wide[:, self.shift:self.shift + self.d] if self.pitch else wide
        if fill is not None:
            v.copy_(fill)
        return v

    def rows(self, dtype, scale=1.0, fill=None):
        return self.empty(dtype, (scale * self.randn(self.T, self.d) if fill is None else fill).to(dtype))

    def post_ref(self, res, y, mag_y=None):
        y64 = f64(y) if isinstance(y, torch.Tensor) else y
        return B.post_fwd(f64(res), y64, np.abs(y64) if mag_y is None else mag_y, self.post,
                          self.q["post_w"], self.q["post_b"], self.q["gate"], self.gate_kind,
                          self.act, self.a, self.b)

    def check_untouched(self, t):
        """Nothing written beside a pitched tensor's rows."""
        if self.pitch and self.T:
            base = t._base
            assert torch.isnan(base[:, :self.shift]).all()
            assert torch.isnan(base[:, self.shift + self.d:]).all()


SHAPES = [dict(T=1, d=64), dict(T=1, d=7168), dict(T=3, d=1), dict(T=5, d=7), dict(T=17, d=31),
          dict(T=130, d=2048), dict(T=9, d=1441), dict(T=4, d=4104), dict(T=3, d=8200),
          dict(T=2, d=16384), dict(T=2, d=16383), dict(T=300, d=256), dict(T=700, d=96),
          dict(T=37, d=520, pitch=8), dict(T=37, d=520, pitch=9, shift=3),
          dict(T=33, d=4096, pitch=24, shift=8), dict(T=1000, d=72),
          dict(T=700, d=2048), dict(T=320, d=7168), dict(T=310, d=9000), dict(T=900, d=1448, pitch=8),
          dict(T=600, d=1001), dict(T=5200, d=256), dict(T=1300, d=1000)]
KINDS = [dict(), dict(pre="layer", bias=True), dict(types="bf16/fp32/fp32", offset=1.0),
         dict(pre="layer", types="fp32/fp32/fp32"), dict(types="bf16/fp32/bf16", weights=False),
         dict(types="fp32/fp32/bf16", bias=True)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("kind", KINDS, ids=str)
def test_pre_norm(shape, kind):
    c = Case(**shape, **kind)
    res = c.rows(c.rt, 2.0)
    x = c.empty(c.at)
    c.m.moe_block_pre_norm_fwd(c.desc, res, c.p["pre_w"], c.p["pre_b"], x)
    ref, mag = B.norm_fwd(f64(res), c.pre, c.q["pre_w"], c.q["pre_b"])
    check("x", x, ref, mag, 128)
    c.check_untouched(x)
    dx, dres_in = c.rows(c.at, 0.1), c.rows(c.rt, 0.1)
    for given in (dres_in, None):
        dres = c.empty(c.rt)
        dw = torch.full((c.d,), 7.0, dtype=c.pt, device="cuda")
        db = torch.full((c.d,), 7.0, dtype=c.pt, device="cuda") if c.p["pre_b"] is not None else None
        c.m.moe_block_pre_norm_bwd(c.desc, dx, res, c.p["pre_w"], given, dres, dw, db, c.ws, 0.75)
        (D, mag), rw, rb = B.join_grads(f64(given), f64(dx), f64(res), c.pre, c.q["pre_w"], 0.75)
        check("dres", dres, D, mag, 128)
        check("dw", dw, *rw, 128 + 192 + c.T)
        if db is not None:
            check("db", db, *rb, 128 + 192 + c.T)
        c.check_untouched(dres)


POSTS = [dict(post="rms"), dict(post="layer", gate="channel", bias=True),
         dict(post="rms", gate="token", act="sigmoid", types="bf16/fp32/fp32"),
         dict(post="layer", gate="full", act="tanh", types="fp32/fp32/fp32", pre="layer"),
         dict(post=None, gate="channel", act="tanh"), dict(post=None, gate="token"),
         dict(post="rms", gate="channel", act="sigmoid", types="bf16/fp32/bf16", bias=True,
              offset=1.0),
         dict(post="rms", gate="full", weights=False), dict(post="layer", gate="token", bias=True)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("kind", POSTS, ids=str)
@pytest.mark.parametrize("next_norm", [True, False])
def test_post_norm(shape, kind, next_norm):
    c = Case(**shape, **kind)
    res, y = c.rows(c.rt, 2.0), c.rows(c.at, 0.7)
    out, x = c.empty(c.rt), c.empty(c.at) if next_norm else None
    c.m.moe_block_post_norm_fwd(c.desc, res, y, c.p, out, x)
    r, mag = c.post_ref(res, y)
    check("res_out", out, r, mag, 128)
    c.check_untouched(out)
    if next_norm:
        check("x", x, *B.norm_fwd_of(r, mag, c.pre, c.q["pre_w"], c.q["pre_b"]), 256)
        c.check_untouched(x)
    # backward from the stored residual
    dres_in = c.rows(c.rt, 0.1)
    dx = c.rows(c.at, 0.1) if next_norm else None
    dres, dy = c.empty(c.rt), c.empty(c.at)
    grads = {}
    for n in ("pre_w", "pre_b", "post_w", "post_b"):
        if c.p[n] is not None and (next_norm or n.startswith("post")):
            grads[n] = torch.full((c.d,), 7.0, dtype=c.pt, device="cuda")
    if c.gate_kind == "channel":
        grads["gate"] = torch.full((c.d,), 7.0, dtype=c.pt, device="cuda")
    elif c.gate_kind == "token":
        grads["gate"] = torch.full((c.T,), 7.0, device="cuda")
    elif c.gate_kind == "full":
        grads["gate"] = c.empty(c.at)
    c.m.moe_block_post_norm_bwd(c.desc, dres_in, dx, out if next_norm else None, y, c.p, dres, dy,
                                grads, c.ws, 0.75)
    (D, mag), dpw, dpb = B.join_grads(f64(dres_in), f64(dx), f64(out), c.pre, c.q["pre_w"], 0.75)
    check("dres", dres, D, mag, 128)
    ref = B.post_bwd(D, mag, f64(y), c.post, c.q["post_w"], c.q["post_b"], c.q["gate"],
                     c.gate_kind, c.act, c.b)
    check("dy", dy, *ref["dy"], 256)
    c.check_untouched(dy)
    rows = 256 + 192 + c.T
    for n, pair in (("pre_w", dpw), ("pre_b", dpb), ("post_w", ref.get("dw")),
                    ("post_b", ref.get("db"))):
        if n in grads:
            check(n, grads[n], *pair, rows)
    if c.gate_kind:
        check("gate", grads["gate"], *ref["gate"], rows)


@pytest.mark.parametrize("k,shape,kind", [
    (1, dict(T=5, d=64), dict()), (4, dict(T=130, d=2880), dict(gate="channel")),
    (6, dict(T=33, d=2048), dict(post="layer", types="bf16/fp32/fp32", bias=True)),
    (3, dict(T=9, d=77), dict(types="fp32/fp32/fp32")), (32, dict(T=3, d=520, pitch=9, shift=1), dict()),
    (2, dict(T=4, d=8200), dict(post=None, gate="token", act="sigmoid")),
    # many rows: the ring, and more expert rows a token than it holds
    (4, dict(T=700, d=2880), dict()), (1, dict(T=700, d=2048), dict(gate="token", act="tanh")),
    (8, dict(T=1300, d=1000), dict(types="bf16/fp32/bf16", gate="full", bias=True)),
    (12, dict(T=400, d=4096), dict()), (2, dict(T=200, d=8200), dict(gate="channel", pre="layer")),
    (6, dict(T=700, d=2048), dict(types="fp32/fp32/fp32", post="layer"))], ids=str)
def test_post_norm_on_expert_rows(k, shape, kind):
    """The combined rows, and the same results as combining first; with and
    without the combined rows written."""
    c = Case(**shape, **kind)
    cap = c.T * k + 13
    Y = (0.7 * c.randn(cap, c.d)).to(c.at).cuda()
    row_of = torch.randperm(cap, generator=c.g)[:c.T * k].to(torch.int32).view(c.T, k).cuda()
    w = torch.softmax(c.randn(c.T, k), dim=1).cuda()
    res = c.rows(c.rt, 2.0)
    out, x, y = c.empty(c.rt), c.empty(c.at), c.empty(c.at)
    c.m.moe_block_post_norm_fwd(c.desc, res, Y, c.p, out, x, dict(row_of=row_of, topk_w=w, y_out=y))
    y64, mag_y = B.combine_rows(f64(Y), row_of.cpu().numpy(), w.cpu().numpy())
    check("y", y, y64, mag_y, 64)
    r, mag = c.post_ref(res, y64, mag_y)
    check("res_out", out, r, mag, 192)
    check("x", x, *B.norm_fwd_of(r, mag, c.pre, c.q["pre_w"], c.q["pre_b"]), 384)
    out2, x2 = c.empty(c.rt), c.empty(c.at)
    c.m.moe_block_post_norm_fwd(c.desc, res, Y, c.p, out2, x2, dict(row_of=row_of, topk_w=w))
    assert torch.equal(out, out2) and torch.equal(x, x2)
    assert c.m.moe_read_device_status() == 0


@pytest.mark.parametrize("T,d", [(6, 256), (1300, 1024)])
def test_expert_rows_out_of_range_are_reported_and_zero(T, d):
    """A row index outside the buffer is not read: the status word says so, and
    the other tokens are as they should be."""
    c = Case(T=T, d=d)
    Y = c.randn(2 * T, d).to(c.at).cuda()
    row_of = torch.arange(2 * T, dtype=torch.int32).view(T, 2).cuda()
    w = torch.full((T, 2), 0.5, device="cuda")
    res = c.rows(c.rt)
    good, bad = c.empty(c.rt), c.empty(c.rt)
    c.m.moe_block_post_norm_fwd(c.desc, res, Y, c.p, good, None, dict(row_of=row_of, topk_w=w))
    assert c.m.moe_read_device_status(clear=True) == 0
    row_of[2, 1], row_of[4, 0] = 2 * T, -1
    c.m.moe_block_post_norm_fwd(c.desc, res, Y, c.p, bad, None, dict(row_of=row_of, topk_w=w))
    torch.cuda.synchronize()
    assert c.m.moe_read_device_status(clear=True) == 0x1
    rest = [0, 1, 3, *range(5, T)]
    assert torch.equal(good[rest], bad[rest])
    only = 0.5 * f64(Y)[4:5]
    r, mag = B.post_fwd(f64(res)[2:3], only, np.abs(only), c.post, c.q["post_w"], None,
                        res_scale=c.a, branch_scale=c.b)
    check("the other slot alone", bad[2:3], r, mag, 128)


def test_no_tokens():
    """T = 0: the forward does nothing, the backward's gradients are zero."""
    c = Case(T=0, d=96, gate="channel", bias=True)
    none = torch.empty(0, 96, dtype=c.at, device="cuda")
    c.m.moe_block_pre_norm_fwd(c.desc, none, c.p["pre_w"], c.p["pre_b"], none)
    c.m.moe_block_post_norm_fwd(c.desc, none, none, c.p, none, none)
    grads = {n: torch.full((96,), 7.0, dtype=c.pt, device="cuda") for n in c.p}
    c.m.moe_block_post_norm_bwd(c.desc, none, none, none, none, c.p, none, none, grads, c.ws)
    for n, t in grads.items():
        assert torch.count_nonzero(t) == 0, n
    dw = torch.full((96,), 7.0, dtype=c.pt, device="cuda")
    c.m.moe_block_pre_norm_bwd(c.desc, none, none, c.p["pre_w"], None, none, dw, None, c.ws)
    assert torch.count_nonzero(dw) == 0


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_rows_of_zeros_constants_and_not_numbers(kind):
    """Zero and constant rows are finite; an Inf or NaN stays in its row."""
    c = Case(T=40, d=264, pre=kind, post=kind, gate="channel", bias=True)
    res, y = c.rows(c.rt), c.rows(c.at)
    clean = c.empty(c.rt), c.empty(c.at)
    c.m.moe_block_post_norm_fwd(c.desc, res, y, c.p, *clean)
    y[3], res[5], y[5] = 0.0, 0.0, 0.0
    y[7], res[7] = 2.5, -1.0
    out, x = c.empty(c.rt), c.empty(c.at)
    c.m.moe_block_post_norm_fwd(c.desc, res, y, c.p, out, x)
    r, mag = c.post_ref(res, y)
    check("res_out", out, r, mag, 128)
    check("x", x, *B.norm_fwd_of(r, mag, c.pre, c.q["pre_w"], c.q["pre_b"]), 256)
    y[11, 4], res[13, 263], y[17, 0] = float("nan"), float("inf"), float("-inf")
    c.m.moe_block_post_norm_fwd(c.desc, res, y, c.p, out, x)
    fine = [t for t in range(40) if t not in (3, 5, 7, 11, 13, 17)]
    assert torch.equal(out[fine], clean[0][fine]) and torch.equal(x[fine], clean[1][fine])
    for t in (11, 13, 17):
        assert torch.isnan(x[t]).any()


def test_large_mean_under_a_layer_norm():
    """The variance is taken about the mean: rows far from zero keep theirs."""
    c = Case(T=8, d=1000, pre="layer", types="fp32/fp32/fp32")
    res = c.rows(c.rt, fill=c.randn(8, 1000) + 3000.0)
    x = c.empty(c.at)
    c.m.moe_block_pre_norm_fwd(c.desc, res, c.p["pre_w"], None, x)
    ref, mag = B.norm_fwd(f64(res), c.pre, c.q["pre_w"], None)
    check("x", x, ref, mag, 128)


@pytest.mark.parametrize("shape", [dict(T=515, d=1024, gate="token", act="sigmoid", bias=True),
                                   dict(T=1700, d=1024, gate="token"),
                                   dict(T=700, d=2049, gate="token", types="fp32/fp32/fp32"),
                                   dict(T=700, d=2048, gate="token", types="bf16/fp32/fp32")], ids=str)
def test_in_place_and_on_another_stream_and_twice(shape):
    """res_out may be res, dres may be dres_in; on a side stream; equal inputs
    give equal bits."""
    c = Case(**shape)
    res, y, dx, dres_in = c.rows(c.rt), c.rows(c.at), c.rows(c.at), c.rows(c.rt)
    out, x = c.empty(c.rt), c.empty(c.at)
    c.m.moe_block_post_norm_fwd(c.desc, res, y, c.p, out, x)
    dres, dy = c.empty(c.rt), c.empty(c.at)

    def grads():
        return {n: torch.empty(c.T if n == "gate" else c.d, dtype=torch.float32 if n == "gate" else c.pt,
                               device="cuda") for n, p in c.p.items() if p is not None}

    g1, g2 = grads(), grads()
    c.m.moe_block_post_norm_bwd(c.desc, dres_in, dx, out, y, c.p, dres, dy, g1, c.ws, 0.75)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dy2, x2 = c.empty(c.at), c.empty(c.at)
    c.m.moe_block_post_norm_fwd(c.desc, res, y, c.p, res, x2, stream=side)
    c.m.moe_block_post_norm_bwd(c.desc, dres_in, dx, res, y, c.p, dres_in, dy2, g2, c.ws, 0.75,
                                stream=side)
    side.synchronize()
    assert torch.equal(res, out) and torch.equal(x2, x)
    assert torch.equal(dres_in, dres) and torch.equal(dy2, dy)
    for n in g1:
        assert torch.equal(g1[n], g2[n]), n


def test_replays_in_a_cuda_graph():
    c = Case(T=200, d=768, gate="channel")
    res, y, dx, dres_in = c.rows(c.rt), c.rows(c.at), c.rows(c.at), c.rows(c.rt)
    new = [t.clone() for t in (c.rows(c.rt), c.rows(c.at))]

    def outs():
        return dict(out=c.empty(c.rt), x=c.empty(c.at), dres=c.empty(c.rt), dy=c.empty(c.at),
                    grads={n: torch.zeros(c.d, dtype=c.pt, device="cuda")
                           for n in ("pre_w", "post_w", "gate")})

    def step(o, stream=None):
        c.m.moe_block_post_norm_fwd(c.desc, res, y, c.p, o["out"], o["x"], stream=stream)
        c.m.moe_block_post_norm_bwd(c.desc, dres_in, dx, o["out"], y, c.p, o["dres"], o["dy"],
                                    o["grads"], c.ws, stream=stream)

    captured, eager = outs(), outs()
    step(captured)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        step(captured, s)
    res.copy_(new[0])
    y.copy_(new[1])
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    step(eager)
    torch.cuda.synchronize()
    for n in ("out", "x", "dres", "dy"):
        assert torch.equal(captured[n], eager[n]), n
    for n, t in eager["grads"].items():
        assert torch.equal(captured["grads"][n], t), n


def test_gradient_against_differences():
    """The kernels' forward, moved a step h to either side along one direction
    of all inputs, against the kernels' gradient.  The bound: the forward's
    rounding over h, plus what a difference of step h leaves by the oracle."""
    c = Case(T=6, d=200, pre="layer", post="rms", gate="channel", act="sigmoid",
             types="fp32/fp32/fp32", bias=True)
    h = 2.0 ** -7
    t = {"res": c.rows(c.rt), "y": c.rows(c.at), **{n: v for n, v in c.p.items()}}
    dirs = {n: torch.randn(v.shape, generator=c.g).cuda() for n, v in t.items()}
    dr, dx = c.rows(c.rt), c.rows(c.at)

    def forward(sign):
        q = {n: v + sign * h * dirs[n] for n, v in t.items()}
        out, x = torch.empty_like(dr), torch.empty_like(dx)
        c.m.moe_block_post_norm_fwd(c.desc, q["res"], q["y"], q, out, x)
        loss = (out.double() * dr.double()).sum() + (x.double() * dx.double()).sum()
        z = {n: f64(v) for n, v in q.items()}
        r, mag = B.post_fwd(z["res"], z["y"], np.abs(z["y"]), c.post, z["post_w"], z["post_b"],
                            z["gate"], "channel", "sigmoid", c.a, c.b)
        xx, mag_x = B.norm_fwd_of(r, mag, c.pre, z["pre_w"], z["pre_b"])
        exact = (r * f64(dr)).sum() + (xx * f64(dx)).sum()
        off = (mag * np.abs(f64(dr))).sum() + (mag_x * np.abs(f64(dx))).sum()
        return float(loss), float(exact), 257 * U * float(off)

    (l1, e1, o1), (l0, e0, o0) = forward(1), forward(-1)
    out, x = torch.empty_like(dr), torch.empty_like(dx)
    c.m.moe_block_post_norm_fwd(c.desc, t["res"], t["y"], c.p, out, x)
    dres, dy = torch.empty_like(dr), torch.empty_like(dx)
    grads = {n: torch.empty(c.d, device="cuda") for n in c.p}
    c.m.moe_block_post_norm_bwd(c.desc, dr, dx, out, t["y"], c.p, dres, dy, grads, c.ws)
    grads = {**grads, "res": c.a * dres, "y": dy}
    inner = sum(float((grads[n].double() * dirs[n].double()).sum()) for n in t)
    r, mag = c.post_ref(t["res"], t["y"])
    (D, magD), dpw, dpb = B.join_grads(f64(dr), f64(dx), r, c.pre, c.q["pre_w"], 1.0)
    ref = B.post_bwd(D, magD, f64(t["y"]), c.post, c.q["post_w"], c.q["post_b"], c.q["gate"],
                     "channel", "sigmoid", c.b)
    ref = {"res": (c.a * D, c.a * magD), "y": ref["dy"], "pre_w": dpw, "pre_b": dpb,
           "post_w": ref["dw"], "post_b": ref["db"], "gate": ref["gate"]}
    exact = sum(float((ref[n][0] * f64(dirs[n])).sum()) for n in t)
    off = sum(float((ref[n][1] * np.abs(f64(dirs[n]))).sum()) for n in t) * (512 + c.T) * U
    bound = (o1 + o0) / (2 * h) + abs((e1 - e0) / (2 * h) - exact) + off
    assert abs((l1 - l0) / (2 * h) - inner) <= bound


def test_rows_past_two_to_the_31_elements():
    """A buffer of more than 2^31 elements: the last rows by 64-bit offsets."""
    T, d, ld = 9, 64, 1 << 28
    c = Case(T=T, d=d)
    base = torch.empty((T, ld), dtype=c.rt, device="cuda")
    res = base[:, 8:8 + d]
    res.copy_(c.randn(T, d).to(c.rt))
    x = torch.empty(T, d, dtype=c.at, device="cuda")
    c.m.moe_block_pre_norm_fwd(c.desc, res, c.p["pre_w"], None, x)
    check("x", x, *B.norm_fwd(f64(res), c.pre, c.q["pre_w"]), 128)
    c.m.moe_block_pre_norm_fwd(c.desc, x, c.p["pre_w"], None, res)
    check("stored far", res, *B.norm_fwd(f64(x), c.pre, c.q["pre_w"]), 128)
