"""The residual block's norms where a group of threads walks down several rows:
every slot of its ring is used again, on plain rows and on expert rows.

A group's rows follow from the launchers' rules: d = 256 has 16 groups a block,
d = 1040 five (two units a thread) or eight (four), one block an SM.  With four
rows for each of the most groups every group has four or more.  Bounds: see
test_gpu_block_norm.py, whose checks run here on these sizes."""
import numpy as np
import pytest
import torch

import oracle.block_oracle as B
import tests.test_gpu_block_norm as norms
from tests.test_gpu_block_norm import Case, U, check, f64

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

GROUPS = {256: 16, 1040: 8}


def size(d):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return dict(T=4 * GROUPS[d] * sms + 37, d=d)


@pytest.mark.parametrize("d", list(GROUPS))
@pytest.mark.parametrize("kind", [dict(), dict(pre="layer", bias=True),
                                  dict(types="bf16/fp32/fp32", offset=1.0),
                                  dict(pre="layer", types="fp32/fp32/fp32")], ids=str)
def test_pre_norm(d, kind):
    norms.test_pre_norm(size(d), kind)


@pytest.mark.parametrize("d", list(GROUPS))
@pytest.mark.parametrize("kind,next_norm", [
    (dict(post="rms", gate="channel"), True), (dict(post="rms"), False),
    (dict(post="rms", gate="token", act="sigmoid", types="bf16/fp32/fp32"), True),
    (dict(post="rms", types="fp32/fp32/fp32"), True),
    (dict(post="layer", pre="layer", gate="channel", bias=True), True),
    (dict(post="layer", gate="full", act="tanh", types="fp32/fp32/fp32", pre="layer"), True),
    (dict(post=None, gate="token"), False)], ids=str)
def test_post_norm(d, kind, next_norm):
    norms.test_post_norm(size(d), kind, next_norm)


# (k, the ring's rows): three, two and one row in the RMS form, which has four
# units a thread; the general form has two; k = 6 has no ring
@pytest.mark.parametrize("k,kind", [
    (1, dict()), (2, dict()), (4, dict(gate="channel")), (2, dict(types="bf16/fp32/fp32")),
    (2, dict(post="layer", pre="layer", bias=True)), (8, dict(post="layer", gate="token")),
    (2, dict(types="fp32/fp32/fp32", post="layer")), (6, dict())], ids=str)
def test_expert_rows(k, kind):
    norms.test_post_norm_on_expert_rows(k, size(1040), kind)


@pytest.mark.parametrize("kind", [dict(), dict(post="layer")], ids=str)
def test_expert_rows_out_of_range(kind):
    """Indexes out of range in a group's first, middle and last rows are counted
    as zero rows; the other tokens' bits do not change."""
    c = Case(**size(1040), **kind)
    T, d, k = c.T, c.d, 2
    Y = c.randn(2 * T, d).to(c.at).cuda()
    row_of = torch.randperm(2 * T, generator=c.g).to(torch.int32).view(T, k).cuda()
    w = torch.softmax(c.randn(T, k), dim=1).cuda()
    res, good, bad = c.rows(c.rt), c.empty(c.rt), c.empty(c.rt)
    c.m.moe_block_post_norm_fwd(c.desc, res, Y, c.p, good, None, dict(row_of=row_of, topk_w=w))
    assert c.m.moe_read_device_status(clear=True) == 0
    at = list(range(3, T, 97))
    other = row_of.clone()
    for i, t in enumerate(at):
        other[t, i % k] = (2 * T, -1, 1 << 30)[i % 3]
    c.m.moe_block_post_norm_fwd(c.desc, res, Y, c.p, bad, None, dict(row_of=other, topk_w=w))
    torch.cuda.synchronize()
    assert c.m.moe_read_device_status(clear=True) == 0x1
    rest = torch.ones(T, dtype=torch.bool)
    rest[at] = False
    rest = rest.cuda()
    assert torch.equal(good[rest], bad[rest])
    kept = np.array([1 - i % k for i in range(len(at))])
    rows = row_of.cpu().numpy()[at, kept][:, None]
    y, mag = B.combine_rows(f64(Y), rows, w.cpu().numpy()[at, kept][:, None])
    r, mag = B.post_fwd(f64(res)[at], y, mag, c.post, c.q["post_w"], None, res_scale=c.a,
                        branch_scale=c.b)
    check("the other slot alone", bad[at], r, mag, 192)


BAD = {5: float("nan"), 1300: float("inf"), 1301: float("-inf"), 4000: float("nan")}


@pytest.mark.parametrize("d", list(GROUPS))
@pytest.mark.parametrize("kind", [dict(), dict(gate="token", types="bf16/fp32/bf16"),
                                  dict(pre="layer", post="layer", gate="channel", bias=True),
                                  dict(pre="layer", post="layer", types="fp32/fp32/fp32")], ids=str)
@pytest.mark.parametrize("where", ["y", "res", "dx", "dres_in"])
def test_not_numbers_stay_in_their_rows(d, kind, where):
    """An Inf or NaN in a row changes no bit of another row, forward or backward,
    where the sums of two rows meet in one as well."""
    c = Case(**size(d), **kind)
    t = dict(res=c.rows(c.rt), y=c.rows(c.at), dx=c.rows(c.at), dres_in=c.rows(c.rt))
    stored = c.rows(c.rt)

    def run():
        o = dict(out=c.empty(c.rt), x=c.empty(c.at), dres=c.empty(c.rt), dy=c.empty(c.at),
                 pre=c.empty(c.rt), x0=c.empty(c.at))
        c.m.moe_block_pre_norm_fwd(c.desc, t["res"], c.p["pre_w"], c.p["pre_b"], o["x0"])
        c.m.moe_block_post_norm_fwd(c.desc, t["res"], t["y"], c.p, o["out"], o["x"])
        r = t["res"] if where == "res" else stored
        c.m.moe_block_post_norm_bwd(c.desc, t["dres_in"], t["dx"], r, t["y"], c.p, o["dres"], o["dy"],
                                    {}, c.ws, 0.75)
        c.m.moe_block_pre_norm_bwd(c.desc, t["dx"], r, c.p["pre_w"], t["dres_in"], o["pre"], None,
                                   None, c.ws, 0.75)
        return o

    stored.copy_(t["res"])
    clean = run()
    for row, v in BAD.items():
        t[where][row, (7 * row) % d] = v
    got = run()
    rest = torch.ones(c.T, dtype=torch.bool)
    rest[list(BAD)] = False
    rest = rest.cuda()
    seen = False
    for n in clean:
        assert torch.isfinite(clean[n]).all(), n
        assert torch.equal(clean[n][rest], got[n][rest]), n
        seen = seen or not torch.isfinite(got[n]).all()
    assert seen


@pytest.mark.parametrize("shape", [dict(T=9, d=1000), dict(T=40, d=1001), dict(T=2, d=16384),
                                   dict(T=5000, d=1040)], ids=str)
def test_layer_norms_far_from_zero(shape):
    """Rows with a mean of 3000 and a spread of 1, forward and backward, on few
    rows and on many."""
    c = Case(**shape, pre="layer", post="layer", types="fp32/fp32/fp32", bias=True)

    def far():
        return c.rows(c.rt, fill=c.randn(c.T, c.d) + 3000.0)

    res, y, dn = far(), far(), c.rows(c.at, 0.1)
    x, out = c.empty(c.at), c.empty(c.rt)
    c.m.moe_block_pre_norm_fwd(c.desc, res, c.p["pre_w"], c.p["pre_b"], x)
    check("x", x, *B.norm_fwd(f64(res), c.pre, c.q["pre_w"], c.q["pre_b"]), 128)
    c.m.moe_block_post_norm_fwd(c.desc, res, y, c.p, out, None)
    check("res_out", out, *c.post_ref(res, y), 128)
    dres, dy = c.empty(c.rt), c.empty(c.at)
    dw, db, dw2 = (torch.empty(c.d, device="cuda") for _ in range(3))
    c.m.moe_block_pre_norm_bwd(c.desc, dn, res, c.p["pre_w"], None, dres, dw, db, c.ws, 0.0)
    c.m.moe_block_post_norm_bwd(c.desc, dn, None, None, y, c.p, None, dy, {"post_w": dw2}, c.ws)

    # dv = rstd (dxh - mean dxh - xhat mean(dxh xhat)): xhat is off by C u times
    # mag (|v| + mean |v|, times rstd), once for each place where it stands; the
    # mean's own error e, at most 96 additions' worth, reaches rstd as e^2 / 2
    def gradient(name, got, scale, v, spec, w, got_w, got_b):
        d = scale * f64(dn)
        xh, mag, rstd = B.norm_stats(f64(v), spec)
        dxh = d * (w + spec.offset)
        (ref, _), rw, rb = B.norm_bwd(d, np.abs(d), f64(v), spec, w)
        s0, s1 = (np.abs(q).mean(axis=1, keepdims=True) for q in (dxh, dxh * xh))
        sm = (np.abs(dxh) * mag).mean(axis=1, keepdims=True)
        terms = rstd * (np.abs(dxh) + s0 + np.abs(xh) * s1)
        off = rstd * (mag * s1 + np.abs(xh) * sm)
        second = 3 * (96 * mag.max()) ** 2 * U           # of terms, in units of u
        check(name, got, ref, terms * (1 + second / 128) + off, 128)
        check(name + " w", got_w, *rw, 128 + 192 + c.T)
        if got_b is not None:
            check(name + " b", got_b, *rb, 128 + 192 + c.T)

    gradient("dres", dres, 1.0, res, c.pre, c.q["pre_w"], dw, db)
    gradient("dy", dy, c.b, y, c.post, c.q["post_w"], dw2, None)
