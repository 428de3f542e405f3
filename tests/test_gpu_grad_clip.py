"""Global gradient norm and clipping on the GPU against the fp64 oracle.

Bounds: squares are summed in fp32 over 32 elements (32 roundings of half a
step and one each for the square, all terms positive) and in fp64 beyond, so
a sum is off by at most 34 * 2^-24 relative, its root by half of that and one
rounding; the clipped value by the factor's error (the norm's and three
roundings) and its own half step."""
import numpy as np
import pytest
import torch

import oracle.block_oracle as B

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

U = 2.0 ** -24
NORM = 18 * U
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


def f64(t):
    return t.detach().double().cpu().numpy()


def measure(tensors, kind="l2", outs=None):
    import moe_expert_mlp_gb300 as m
    g = m.GradList(tensors, outs)
    norm = torch.full((1,), -7.0, device="cuda")
    norms = torch.full((len(tensors),), -7.0, device="cuda")
    ws = torch.full((m.moe_grad_norm_workspace_size(len(tensors)),), 255, dtype=torch.uint8,
                    device="cuda")
    m.moe_grad_norm(g, norm, norms, kind, ws)
    alone = torch.empty_like(norm)
    m.moe_grad_norm(g, alone, None, kind, ws)
    assert torch.equal(alone.view(torch.int32), norm.view(torch.int32))
    return m, g, norm, norms


def check_norms(tensors, kind, norm, norms):
    total, each = B.grad_norm([f64(t) for t in tensors], kind)
    got, parts = float(norm), f64(norms)
    if kind == "inf":
        assert got == total and np.array_equal(parts, each)
    else:
        assert abs(got - total) <= NORM * total, (got, total)
        assert np.all(np.abs(parts - each) <= NORM * each)


def make(shapes, dtype, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(scale * torch.randn(s, generator=g)).to(dtype).cuda() for s in shapes]


SHAPES = {
    "one": [(1,)], "odd": [(7,), (33, 5), (1,), (16385,), (3, 1, 129)],
    "tiles": [(16384,), (16383,), (16385,), (32768,), (5,)],
    "many": [(1 + 37 * i % 301,) for i in range(300)],
    "over_a_launch": [(3 + i % 5, 7) for i in range(1000)],
    "large": [(64, 513, 257), (8, 96), (1 << 20,)],
    "empties": [(0,), (9,), (4, 0), (2, 3), (0, 0)], "all_empty": [(0,), (3, 0)], "none": [],
}


@pytest.mark.parametrize("name", list(SHAPES))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["l2", "inf"])
def test_norm(name, dtype, kind):
    t = make(SHAPES[name], dtype)
    _, _, norm, norms = measure(t, kind)
    check_norms(t, kind, norm, norms)


def check_clipped(outs, grads, norm, max_norm, eps=1e-6):
    f = B.clip_factor(float(norm), max_norm, eps)     # of the kernel's own norm
    for i, (o, g) in enumerate(zip(outs, grads)):
        ref = f64(g) * f
        bound = HALF[o.dtype] * np.abs(ref) + 4 * U * np.abs(ref) + 1e-40
        assert np.all(np.abs(f64(o) - ref) <= bound), i


@pytest.mark.parametrize("name", ["one", "odd", "tiles", "over_a_launch", "large", "empties", "none"])
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32"),
                                   ("fp32", "bf16")])
@pytest.mark.parametrize("max_norm", [0.5, 1e9, 0.0])
def test_clip_into_other_tensors(name, types, max_norm):
    dt = {"bf16": torch.bfloat16, "fp32": torch.float32}
    t = make(SHAPES[name], dt[types[0]], seed=1)
    keep = [v.clone() for v in t]
    outs = [torch.full(v.shape, 7.0, dtype=dt[types[1]], device="cuda") for v in t]
    m, g, norm, _ = measure(t, "l2", outs)
    m.moe_clip_grads(g, norm, max_norm)
    check_clipped(outs, t, norm, max_norm)
    for a, b in zip(t, keep):
        assert torch.equal(a, b)


def test_clip_in_place():
    t = make(SHAPES["odd"], torch.float32, seed=2)
    before = [v.clone() for v in t]
    m, g, norm, _ = measure(t)
    m.moe_clip_grads(g, norm, 0.25)
    check_clipped(t, before, norm, 0.25)
    again = [v.clone() for v in t]
    m.moe_clip_grads(g, torch.full((1,), 0.1, device="cuda"), 0.25)     # below the limit
    for a, b in zip(t, again):
        assert torch.equal(a, b)


def test_mixed_types_and_views():
    """fp32 and bf16 in one list; column slices, transposes, odd starts."""
    base = make([(40, 96), (31, 200), (1000,), (17, 300), (20000, 3)], torch.float32, seed=3)
    low = [b.to(torch.bfloat16) for b in base]
    t = [base[0][:, 3:50], low[1][2:9], base[2][1:], low[2][3:], low[3].t(), base[3][:, ::2],
         low[0][:, 7], low[4][:, :2], base[1][:, 8:136]]
    _, _, norm, norms = measure(t)
    check_norms(t, "l2", norm, norms)
    outs = [torch.full((v.shape[0], v.shape[1] + 5), 7.0, device="cuda")[:, 2:2 + v.shape[1]]
            if v.dim() == 2 and v.stride(1) == 1 else torch.empty_like(v) for v in t]
    m, g, norm, _ = measure(t, "l2", outs)
    m.moe_clip_grads(g, norm, 1.0)
    check_clipped(outs, t, norm, 1.0)
    for o in outs:
        if o._base is not None:
            assert (o._base[:, :2] == 7.0).all() and (o._base[:, 2 + o.shape[1]:] == 7.0).all()


@pytest.mark.parametrize("scale", [1e-22, 1e-30, 3e-41, 1e18, 2e19, 3e36])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_squares_outside_fp32(scale, dtype):
    """Squares that vanish or overflow in fp32 are summed in fp64."""
    t = make([(5000,), (33, 7)], dtype, seed=4, scale=scale)
    t.append(torch.zeros(40, dtype=dtype, device="cuda"))
    _, _, norm, norms = measure(t)
    total, each = B.grad_norm([f64(v) for v in t])
    step = 2.0 ** -149                                   # fp32's smallest, where norms end
    assert abs(float(norm) - total) <= NORM * total + step
    assert np.all(np.abs(f64(norms) - each) <= NORM * each + step)


def test_not_numbers():
    for kind in ("l2", "inf"):
        t = make([(300,), (5000,)], torch.float32, seed=5)
        t[1][4321] = float("inf")
        m, g, norm, norms = measure(t, kind)
        assert float(norm) == np.inf and float(norms[1]) == np.inf and np.isfinite(float(norms[0]))
        m.moe_clip_grads(g, norm, 1.0)                    # a factor of 0
        assert (t[0] == 0).all() and torch.isnan(t[1][4321]) and (t[1][:4321] == 0).all()
        t = make([(300,), (5000,)], torch.bfloat16, seed=5)
        t[0][17], t[1][3] = float("nan"), float("inf")
        m, g, norm, norms = measure(t, kind)
        assert np.isnan(float(norm)) and np.isnan(float(norms[0])) and float(norms[1]) == np.inf
        m.moe_clip_grads(g, norm, 1.0)
        assert torch.isnan(t[0]).all() and torch.isnan(t[1]).all()


def test_replaced_memory_is_seen():
    """A list whose tensor got new memory measures the new one."""
    t = make([(100,), (200,)], torch.float32, seed=6)
    m, g, norm, norms = measure(t)
    old = t[1].data
    t[1].data = 2 * old.clone()
    ws = torch.empty(m.moe_grad_norm_workspace_size(2), dtype=torch.uint8, device="cuda")
    m.moe_grad_norm(g, norm, norms, "l2", ws)
    check_norms(t, "l2", norm, norms)


def test_graph_replay_and_side_stream():
    t = make([(5000,), (64, 33), (200000,)], torch.bfloat16, seed=7)
    outs = [torch.empty(v.shape, device="cuda") for v in t]
    m, g, norm, norms = measure(t, "l2", outs)
    ws = torch.empty(m.moe_grad_norm_workspace_size(3), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        m.moe_grad_norm(g, norm, norms, "l2", ws, stream=s)
        m.moe_clip_grads(g, norm, 1.0, stream=s)
    for v in t:
        v.mul_(3.0)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    check_norms(t, "l2", norm, norms)
    check_clipped(outs, t, norm, 1.0)
    first = norm.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    m.moe_grad_norm(g, norm, norms, "l2", ws, stream=side)
    side.synchronize()
    assert torch.equal(first, norm)


def test_tensor_past_two_to_the_32_elements():
    """More than 2^32 elements in one tensor: its last ones count, and are
    clipped."""
    n = (1 << 32) + 100
    t = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    t[-3:] = 2.0
    t[5] = 2.0
    m, g, norm, _ = measure([t])
    assert float(norm) == 4.0
    m.moe_clip_grads(g, norm, 2.0, 0.0)
    assert t[-3:].tolist() == [1.0] * 3 and float(t[5]) == 1.0 and float(t[1 << 31]) == 0.0
