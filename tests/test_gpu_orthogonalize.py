"""Orthogonalised updates on the GPU: against the oracle with the kernels'
roundings, and against the formula in 64 bits.

Bounds, in the 2-norm of the result.  Beside the oracle's roundings the kernels
add products in fp32: each sum of up to n terms is off by about sqrt(n) 2^-24, so
of the values that are then rounded to fp16 a share of sqrt(n) 2^-24 / 2^-12
falls to the other side of a border, by 2^-11: for n = 4096 a share of 1.6e-2, that
is sqrt(1.6e-2) 2^-11 = 6e-5 in the 2-norm for each of three roundings a step.
Five steps, the last ones counting (the map multiplies an error by up to 3.4 on
the way to one and by up to 1.6 there), come to 6e-5 sqrt(3) (1 + 1.6 + 2.6 + 5 +
10) < 2.2e-3 at the very worst and a third of that where signs differ: MODEL =
1e-3.  bf16's rounding is within 2^-8 of each value.  Against the formula the
fp16 operands' cost is added, as the rounded oracle has it for the same input."""
import math

import numpy as np
import pytest
import torch

import oracle.training_oracle as O

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

MODEL = 1e-3
BF16 = 2.0 ** -8


def f64(t):
    return t.detach().double().cpu().numpy()


def wide_view(shape, dtype, pitched, align=8):
    """A zeroed stack, or a view inside a wider one whose surroundings are 77."""
    if not pitched:
        return torch.zeros(shape, dtype=dtype, device="cuda"), None
    b, r, c = shape
    room = torch.full((b, r + 3, c + 2 * align + 1 - c % 2), 77.0, dtype=dtype, device="cuda")
    return room[:, 1:1 + r, align:align + c], room


def untouched(view, room):
    if room is None:
        return True
    copy = room.clone()
    b, r, c = view.shape
    off = view.storage_offset() - room.stride(1)
    copy[:, 1:1 + r, off:off + c] = 77.0
    return bool((copy == 77.0).all())


def values(shape, kind, seed):
    rng = np.random.default_rng(seed)
    b, r, c = shape
    out = np.zeros(shape)
    for i in range(b):
        if kind == "full":
            out[i] = rng.standard_normal((r, c))
        elif kind == "few tokens":
            out[i] = rng.standard_normal((r, 3)) @ rng.standard_normal((3, c))
        elif kind == "falling":
            out[i] = rng.standard_normal((r, c)) * np.arange(1, c + 1) ** -1.0
        if kind == "mixed":
            out[i] = [rng.standard_normal((r, c)), np.zeros((r, c)), 1e-12 * rng.standard_normal((r, c)),
                      rng.standard_normal((r, 2)) @ rng.standard_normal((2, c))][i % 4]
    return out


def run(g, steps=5, scale=1.0, dtype=torch.bfloat16, mom=None, momentum=0.0, dampening=0.0,
        nesterov=False, pitched=False, in_place=False, coefficients=O.DEFAULT, eps=1e-7,
        align=8, stream=None):
    import moe_expert_mlp_gb300 as m
    shape = g.shape
    name = "fp32" if dtype is torch.float32 else "bf16"
    desc = m.make_orthogonalize_desc(*shape, grad_dtype=name, steps=steps, coefficients=coefficients,
                                     eps=eps, momentum=momentum, dampening=dampening,
                                     nesterov=nesterov, scale=scale)
    grad, _ = wide_view(shape, dtype, pitched, align)
    grad.copy_(torch.from_numpy(g))
    out, out_room = wide_view(shape, torch.bfloat16, pitched, align)
    mi = mo = mo_room = None
    if mom is not None:
        mi, mo_room = wide_view(shape, torch.float32, pitched, align)
        mi.copy_(torch.from_numpy(mom))
        mo = mi
        if not in_place:
            mo, mo_room = wide_view(shape, torch.float32, pitched, align)
    ws = torch.full((m.moe_orthogonalize_workspace_size(desc),), 255, dtype=torch.uint8, device="cuda")
    before = None if mom is None else mi.clone()
    m.moe_orthogonalize(desc, grad, out, ws, mi, mo, stream)
    torch.cuda.synchronize()
    assert m.moe_read_device_status() == 0
    assert untouched(out, out_room)
    if mom is not None:
        assert untouched(mo, mo_room)
    return f64(grad), (None if before is None else f64(before)), f64(out), (
        None if mo is None else f64(mo))


def joined(shape, steps):
    """Whether the kernels take the first two steps as one."""
    b, r, c = shape
    m, n = sorted((r, c))
    tiles = -(-m // 256)
    return m > 128 and steps >= 5 and n >= 2 * m and b * tiles * (tiles + 1) // 2 >= 128


def check(grad, mom, out, mom_out, steps=5, scale=1.0, momentum=0.0, dampening=0.0, nesterov=False,
          coefficients=O.DEFAULT, eps=1e-7):
    for i in range(len(grad)):
        m2, u = O.momentum_update(grad[i], None if mom is None else mom[i], momentum, dampening,
                                  nesterov)
        if mom is not None:
            mag = abs(momentum) * np.abs(mom[i]) + abs(1 - dampening) * np.abs(grad[i])
            assert np.all(np.abs(mom_out[i] - m2) <= 6 * O.U32 * mag + 1e-44)
        ref = O.orthogonalize(u, steps, coefficients, eps, scale)
        rounded = O.orthogonalize_rounded(u, steps, coefficients, eps, scale,
                                          joined(grad.shape, steps))
        size = np.linalg.norm(ref)
        if size == 0:
            assert not out[i].any()
            continue
        assert np.linalg.norm(out[i] - rounded) <= (MODEL + BF16) * size, i
        cost = np.linalg.norm(rounded - ref)
        assert np.linalg.norm(out[i] - ref) <= cost + (MODEL + BF16) * size, i


SHAPES = [(1, 1, 1), (2, 1, 9), (2, 7, 1), (1, 16, 16), (3, 64, 64), (1, 64, 300), (1, 300, 64),
          (2, 100, 129), (1, 128, 128), (2, 128, 1000), (1, 1000, 130), (1, 256, 256), (4, 255, 257),
          (2, 257, 255), (1, 256, 2048), (1, 2048, 256), (2, 320, 600), (1, 600, 520), (1, 513, 1025),
          (1, 1441, 1001)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_shapes(shape, dtype):
    check(*run(values(shape, "full", 1), dtype=dtype))


@pytest.mark.parametrize("shape", [(8, 96, 200), (8, 200, 96), (4, 300, 300), (4, 64, 2048),
                                   (4, 700, 264)])
@pytest.mark.parametrize("kind", ["few tokens", "falling", "mixed"])
def test_spectra(shape, kind):
    check(*run(values(shape, kind, 2), scale=0.2), scale=0.2)


@pytest.mark.parametrize("shape", [(2, 72, 136), (2, 130, 61), (3, 300, 513), (1, 520, 264)])
@pytest.mark.parametrize("steps", [1, 2, 3, 4])
def test_steps(shape, steps):
    check(*run(values(shape, "full", 3), steps=steps), steps=steps)


@pytest.mark.parametrize("coefficients,steps", [((1.5, -0.5, 0.0), 12), ((2.0, -1.5, 0.5), 6),
                                                ((1.0, 0.0, 0.0), 2)])
@pytest.mark.parametrize("shape", [(2, 80, 112), (1, 400, 300)])
def test_coefficients(shape, coefficients, steps):
    kw = dict(coefficients=coefficients, steps=steps)
    check(*run(values(shape, "full", 4), **kw), **kw)


@pytest.mark.parametrize("shape", [(3, 64, 192), (2, 101, 77), (2, 300, 401), (1, 640, 512)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("nesterov,in_place,pitched", [(False, False, False), (True, True, False),
                                                       (True, False, True), (False, True, True)])
def test_momentum(shape, dtype, nesterov, in_place, pitched):
    g = values(shape, "full", 5)
    m = values(shape, "few tokens", 6) * 0.5
    kw = dict(momentum=0.9, dampening=0.1, nesterov=nesterov)
    check(*run(g, dtype=dtype, mom=m, in_place=in_place, pitched=pitched, **kw), **kw)


@pytest.mark.parametrize("align", [1, 4, 8])
@pytest.mark.parametrize("shape", [(2, 65, 128), (2, 128, 63), (2, 300, 264)])
def test_unaligned_rows(shape, align):
    check(*run(values(shape, "full", 7), pitched=True, align=align))


def test_momentum_of_zero_is_kept_too():
    g = values((2, 96, 96), "full", 8)
    check(*run(g, mom=values((2, 96, 96), "full", 9)))


@pytest.mark.parametrize("scale", [1e-22, 1e-6, 1e16])
@pytest.mark.parametrize("shape", [(2, 64, 80), (1, 300, 280)])
def test_size_of_the_gradient_does_not_matter(shape, scale):
    """eps far below the norm; the squares of 1e-22 leave fp32's range."""
    g = values(shape, "full", 10) * scale
    check(*run(g, dtype=torch.float32, eps=1e-30), eps=1e-30)


@pytest.mark.parametrize("shape", [(3, 48, 90), (3, 300, 270)])
def test_inf_and_nan_stay_in_their_matrix(shape):
    g = values(shape, "full", 11)
    clean = run(g)[2]
    g[1, 5, 7] = np.nan
    out = run(g)[2]
    assert np.isnan(out[1]).all()
    assert np.array_equal(out[[0, 2]], clean[[0, 2]])
    g[1, 5, 7] = np.inf
    out = run(g)[2]
    assert np.isnan(out[1]).all() and np.array_equal(out[[0, 2]], clean[[0, 2]])


@pytest.mark.parametrize("shape", [(2, 64, 100), (5, 270, 530)])
def test_results_repeat_and_zero_rows_stay_zero(shape):
    g = values(shape, "full", 12)
    g[:, 3::5] = 0
    first, again = run(g)[2], run(g)[2]
    assert np.array_equal(first, again) and not first[:, 3::5].any()


def test_one_matrix_of_two_dimensions_over_its_own_gradient():
    import moe_expert_mlp_gb300 as m
    g = torch.from_numpy(values((1, 70, 150), "full", 13)[0]).to("cuda", torch.bfloat16)
    keep = f64(g)
    desc = m.make_orthogonalize_desc(1, 70, 150)
    ws = torch.empty(m.moe_orthogonalize_workspace_size(desc), dtype=torch.uint8, device="cuda")
    m.moe_orthogonalize(desc, g, g, ws)
    check(keep[None], None, f64(g)[None], None)


def test_no_matrices():
    import moe_expert_mlp_gb300 as m
    desc = m.make_orthogonalize_desc(0, 70, 150)
    ws = torch.empty(m.moe_orthogonalize_workspace_size(desc), dtype=torch.uint8, device="cuda")
    g = torch.empty((0, 70, 150), dtype=torch.bfloat16, device="cuda")
    m.moe_orthogonalize(desc, g, g.clone(), ws)


@pytest.mark.parametrize("shape", [(2, 64, 256), (2, 300, 520)])
def test_graph_on_another_stream(shape):
    import moe_expert_mlp_gb300 as m
    desc = m.make_orthogonalize_desc(*shape, momentum=0.9, nesterov=True)
    ws = torch.empty(m.moe_orthogonalize_workspace_size(desc), dtype=torch.uint8, device="cuda")
    g = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    mom = torch.zeros(shape, device="cuda")
    out = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    m.moe_orthogonalize(desc, g, out, ws, mom, stream=stream)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        m.moe_orthogonalize(desc, g, out, ws, mom)
    for seed in (1, 2):
        g.copy_(torch.from_numpy(values(shape, "full", seed)))
        before = f64(mom)
        graph.replay()
        torch.cuda.synchronize()
        check(f64(g), before, f64(out), f64(mom), momentum=0.9, nesterov=True)


@pytest.mark.parametrize("shape", [(43, 300, 640), (43, 610, 300), (130, 140, 300)])
@pytest.mark.parametrize("kind,steps", [("full", 5), ("few tokens", 5), ("mixed", 6), ("falling", 5)])
def test_first_two_steps_as_one(shape, kind, steps):
    assert joined(shape, steps)
    check(*run(values(shape, kind, 15), steps=steps, scale=0.3), steps=steps, scale=0.3)


def test_many_small_matrices():
    check(*run(values((200, 24, 40), "mixed", 14)))


# clusters of one to eight, whose shares of 64 or 128 rows are not all alike
@pytest.mark.parametrize("shape", [(3, 50, 61), (3, 64, 100), (3, 50, 150), (2, 64, 250), (2, 64, 300),
                                   (2, 33, 384), (2, 64, 448), (2, 17, 500), (2, 100, 80), (2, 128, 129),
                                   (2, 128, 160), (2, 90, 190), (2, 128, 224), (2, 65, 256)])
@pytest.mark.parametrize("tall", [False, True])
def test_small_matrices_of_every_cluster(shape, tall):
    b, m, n = shape
    check(*run(values((b, n, m) if tall else shape, "full", 21)))


@pytest.mark.parametrize("shape", [(20, 64, 512), (6, 128, 900), (8, 256, 512), (3, 520, 700), (43, 300, 640)])
def test_many_runs_give_equal_bits(shape):
    import moe_expert_mlp_gb300 as m
    g = torch.from_numpy(values(shape, "full", 22)).cuda().bfloat16()
    desc = m.make_orthogonalize_desc(*shape)
    ws = torch.empty(m.moe_orthogonalize_workspace_size(desc), dtype=torch.uint8, device="cuda")
    first, out = torch.empty_like(g), torch.empty_like(g)
    m.moe_orthogonalize(desc, g, first, ws)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(40):
        m.moe_orthogonalize(desc, g, out.zero_(), ws)
        differ += (out != first).sum()
    assert int(differ) == 0 and m.moe_read_device_status() == 0


def test_two_calls_at_once_and_graphs_that_share_a_workspace():
    """Calls on two streams with a workspace each, large (every SM) and small; then
    two graphs over one workspace, replayed in turn."""
    import moe_expert_mlp_gb300 as m
    shapes = [(4, 300, 700), (2, 520, 400), (8, 64, 512)]
    calls = []
    for i, shape in enumerate(shapes):
        g = torch.from_numpy(values(shape, "full", 30 + i)).cuda().bfloat16()
        desc = m.make_orthogonalize_desc(*shape)
        ws = torch.empty(m.moe_orthogonalize_workspace_size(desc), dtype=torch.uint8, device="cuda")
        alone, out = torch.empty_like(g), torch.zeros_like(g)
        m.moe_orthogonalize(desc, g, alone, ws)
        calls.append((desc, g, out, ws, alone))
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, (desc, g, out, ws, _) in zip(streams, calls):
            m.moe_orthogonalize(desc, g, out, ws, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(out, alone) for _, _, out, _, alone in calls)
    ws = max((c[3] for c in calls), key=lambda t: t.numel())
    graphs = []
    for desc, g, out, _, _ in calls:
        out.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            m.moe_orthogonalize(desc, g, out, ws)
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out, alone) for _, _, out, _, alone in calls)
    assert m.moe_read_device_status() == 0


@pytest.mark.parametrize("shape", [(1, 64, 600), (2, 40, 833), (1, 64, 1000), (2, 128, 900), (1, 70, 1900),
                                   (1, 128, 2048), (3, 17, 4096)])
@pytest.mark.parametrize("tall", [False, True])
def test_small_matrices_of_up_to_sixteen_ctas(shape, tall):
    """Among them clusters in which the last CTAs have no rows of A to add up."""
    b, m, n = shape
    check(*run(values((b, n, m) if tall else shape, "full", 23)))
