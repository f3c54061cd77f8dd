"""What the layer refuses before it enqueues anything (no GPU)."""
import pytest
import torch


@pytest.mark.parametrize("columns", [3, 5, 8])
def test_logits_of_another_number_of_experts(columns):
    """Ids past the weights' experts would have no rows, and the gradient another shape than the logits."""
    import combine_moe_route_gb300 as moe
    w = moe.ExpertWeights.quantized(torch.ones((4, 256, 128)), torch.ones((4, 128, 128)))
    x = torch.zeros((6, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="4 experts"):
        moe.expert_layer(x, torch.zeros((6, columns)), [6], 2, w)
    with pytest.raises(ValueError, match="4 experts"):
        moe.expert_layer(x, torch.zeros(6 * 4), [6], 2, w)
