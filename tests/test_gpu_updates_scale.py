"""The scale of the experts' updates where the packed FC1 has padding rows."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_block_norm import f64
from tests.test_gpu_orthogonalize import check as check_updates
from tests.test_gpu_training_step import SMALL, WL, make
from workloads import scaled

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def by_sides(rows, cols):
    return 0.2 * math.sqrt(max(rows, cols))


@pytest.mark.parametrize("wl", [WL, SMALL, scaled(SMALL, act="srelu")])
def test_scale_without_the_padding(wl):
    """With padding=False, by default and by a function, from the weights' own rows."""
    m, block, res, logits, bias, dres, mask, offsets = make(wl, losses=False)
    layer = block.layer
    rows = 2 * layer.F if layer.gated else layer.F
    want = [np.float32(by_sides(rows, layer.d)), np.float32(by_sides(layer.d, layer.F))]
    asked = []

    def scale(rows, cols):
        asked.append((rows, cols))
        return by_sides(rows, cols)

    block.orthogonal_updates(scale=scale, padding=False)
    assert asked == [(rows, layer.d), (layer.d, layer.F)]
    assert [d.scale for d in block.updates.descs] == want
    updates = block.orthogonal_updates(momentum=0.0, padding=False)
    assert [d.scale for d in updates.descs] == want
    block.step(res, logits, bias, dres)
    torch.cuda.synchronize()
    for g, out, by in zip((layer.dw1p, layer.dw2), updates.outs, want):
        check_updates(f64(g), None, f64(out), None, scale=by)


def test_sizes_are_one_for_each_gradient():
    import moe_expert_mlp_gb300 as m
    g = [torch.zeros(3, 4, device="cuda"), torch.zeros(2, 5, 6, device="cuda")]
    u = m.OrthogonalUpdates(g, momentum=0.0, sizes=[(2, 4), (5, 6)])
    assert [d.scale for d in u.descs] == [np.float32(by_sides(2, 4)), np.float32(by_sides(5, 6))]
    with pytest.raises(ValueError, match="sizes"):
        m.OrthogonalUpdates(g, sizes=[(3, 4)])
    with pytest.raises(ValueError, match="gradient 1"):
        m.OrthogonalUpdates(g, sizes=[(3, 4), (6, 6)])
