"""The feed-forward block carries no autograd graph, and says so where a gradient would
be lost (CPU only: the refusal comes before the device is looked at)."""
import pytest
import torch


@pytest.fixture()
def layer():
    import sparse_mixture_experts_24_b200 as m
    layer = m.MoELayer(2, 1, 64, 64, "bf16")
    yield layer
    layer.close()


@pytest.mark.parametrize("name", ["x", "w1", "w3", "w2"])
def test_a_gradient_that_would_be_lost_is_refused(layer, name):
    import sparse_mixture_experts_24_b200 as m
    t = dict(x=torch.zeros(4, 64, dtype=torch.bfloat16), **{k: torch.zeros(2, 64, 64, dtype=torch.bfloat16)
                                                            for k in ("w1", "w3", "w2")})
    t[name].requires_grad_()
    with pytest.raises(m.MoEError) as ei:
        layer.ffn_forward(**t)
    assert ei.value.status == m.MOE_ERR_INVALID_ARG
    assert "%s requires a gradient" % name in str(ei.value) and "ffn_backward" in str(ei.value)
    # where autograd records nothing there is nothing to lose: the next check answers
    with torch.no_grad(), pytest.raises(m.MoEError) as ei:
        layer.ffn_forward(**t)
    assert "not a CUDA tensor" in str(ei.value)


def test_inside_an_autograd_function_the_call_goes_through(layer):
    """Function.forward runs without recording, so a user's own Function around the two
    calls meets the next check (no GPU here), not the refusal."""
    import sparse_mixture_experts_24_b200 as m

    class Block(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w1, w3, w2):
            return layer.ffn_forward(x, w1, w3, w2)

    w = torch.zeros(2, 64, 64, dtype=torch.bfloat16, requires_grad=True)
    with pytest.raises(m.MoEError) as ei:
        Block.apply(torch.zeros(4, 64, dtype=torch.bfloat16), w, w, w)
    assert "not a CUDA tensor" in str(ei.value)
