"""Host side of a layer with the router's losses, without a GPU: a call that is
refused has enqueued nothing."""
import pytest
import torch


@pytest.fixture
def layer_of(monkeypatch):
    from moe_expert_mlp_gb300.build import build_library
    build_library()
    import moe_expert_mlp_gb300 as m
    m.lib()
    calls = []
    for name in ("moe_route_permute", "moe_route_permute_mx", "moe_route_permute_fused",
                 "moe_router_loss_fwd"):
        monkeypatch.setattr(m._lib, name, lambda *a, name=name, **k: calls.append(name))

    def of(**kw):
        return m.MoEExpertMLP(4, 64, 64, T=8, k=2, device="cpu", **kw), calls

    return of


@pytest.mark.parametrize("given", ["mask", "seq_offsets"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32", "mxfp8", "nvfp4"])
def test_losses_inputs_without_losses_are_refused_before_the_routing(layer_of, dtype, given):
    layer, calls = layer_of(dtype=dtype)
    x, logits = torch.zeros(8, 64), torch.zeros(8, 4)
    kw = {given: torch.ones(8, dtype=torch.bool) if given == "mask" else
          torch.tensor([0, 8], dtype=torch.int32)}
    with pytest.raises(ValueError, match="coefficients"):
        layer.route(x, logits, **kw)
    with pytest.raises(ValueError, match="coefficients"):
        layer.route_fused(x, torch.zeros(4, 64), logits_out=logits, **kw)
    assert calls == []
    layer.route(x, logits)
    assert len(calls) == 1


def test_the_losses_follow_the_routing(layer_of):
    layer, calls = layer_of(balance_coef=0.1)
    layer.route(torch.zeros(8, 64), torch.zeros(8, 4), mask=torch.ones(8, dtype=torch.bool))
    assert calls == ["moe_route_permute", "moe_router_loss_fwd"]


def test_a_block_refuses_them_before_its_norm(layer_of, monkeypatch):
    import moe_expert_mlp_gb300 as m
    layer, calls = layer_of()
    monkeypatch.setattr(m._lib, "GradList", list)
    monkeypatch.setattr(m._lib, "moe_block_pre_norm_fwd", lambda *a: calls.append("norm"))
    block = m.MoEResidualBlock(layer)
    with pytest.raises(ValueError, match="coefficients"):
        block.forward(torch.zeros(8, 64), torch.zeros(8, 4), mask=torch.ones(8, dtype=torch.bool))
    assert calls == []
