"""Lists of gradients on the GPU: what a list measures and writes when its
tensors change.  Bound of a norm: chains of at most 17 squares and three joins in
fp32 before fp64 are 21 roundings of the sum, 11.5 * 2^-24 of its root; the checks
of test_gpu_grad_clip.py allow 18."""
import pytest
import torch

from tests.test_gpu_grad_clip import check_clipped, check_norms, measure

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.mark.parametrize("change", [lambda b: b[:3000], lambda b: b.view(125, 40)[:, :24],
                                    lambda b: b[:5000:2],
                                    lambda b: b.view(torch.bfloat16)[:5000]],
                         ids=["shorter", "rows", "every_other", "other_type"])
def test_a_tensor_changed_at_its_address(change):
    """Norm and clip are those of the tensor as it is now; nothing beside it is
    written."""
    g = torch.Generator().manual_seed(8)
    base = torch.randn(5000, generator=g).to(torch.bfloat16).float().cuda()
    still = torch.randn(300, generator=g).cuda()
    t = base[:]
    m, lst, norm, norms = measure([still, t])
    t.data = change(base)
    before, inside = [still.clone(), t.clone()], torch.zeros(5000, dtype=torch.bool)
    view = change(torch.arange(5000, dtype=torch.float32))
    if view.dtype == torch.float32:
        inside[view.long().flatten()] = True
    else:
        inside[:2500] = True
    ws = torch.empty(m.moe_grad_norm_workspace_size(2), dtype=torch.uint8, device="cuda")
    m.moe_grad_norm(lst, norm, norms, "l2", ws)
    check_norms([still, t], "l2", norm, norms)
    whole = base.clone()
    m.moe_clip_grads(lst, norm, 0.5)
    check_clipped([still, t], before, norm, 0.5)
    assert torch.equal(base[~inside.cuda()], whole[~inside.cuda()])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_norms_do_not_depend_on_where_the_clipped_go(dtype):
    """The same gradients have the same bits of norm in place, with outs in
    wider buffers, and with a description whose out was never set."""
    g = torch.Generator().manual_seed(9)
    t = [torch.randn(400, 300, generator=g).to(dtype).cuda() for _ in range(40)]
    _, lst, norm, norms = measure(t)
    wide = [torch.empty(400, 308, device="cuda")[:, :300] for _ in t]
    m, _, norm2, norms2 = measure(t, "l2", wide)
    assert torch.equal(norm, norm2) and torch.equal(norms, norms2)
    ws = torch.empty(m.moe_grad_norm_workspace_size(len(t)), dtype=torch.uint8, device="cuda")
    for a in lst.array:
        a.rows, a.cols, a.ld = 400, 300, 300
    for out, ld_out, kind in ((None, 0, 0), (1 << 20, 12345, 77)):
        for a in lst.array:
            a.out, a.ld_out, a.out_dtype = out, ld_out, kind
        norm2, norms2 = torch.empty_like(norm), torch.empty_like(norms)
        m._lib.binding().grad_norm(lst.array, len(t), 0, norm2, norms2, ws, None)
        assert torch.equal(norm, norm2) and torch.equal(norms, norms2)
