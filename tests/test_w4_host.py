"""The 4-bit quantiser's binding without a GPU: a group that is none is refused as the
library refuses it."""
import pytest
import torch

import mixture_experts_routing_gb300 as moe


@pytest.fixture(scope="module", autouse=True)
def library():
    from mixture_experts_routing_gb300 import _build
    _build.build()


@pytest.mark.parametrize("group", [0, -32])
def test_quantiser_refuses_a_group_of_no_columns(group):
    m = torch.zeros((4, 128), dtype=torch.bfloat16)
    with pytest.raises(moe.MoEError) as e:
        moe.w4_quantize(m, group, torch.zeros((4, 64), dtype=torch.uint8), torch.zeros((4, 1), dtype=torch.bfloat16))
    assert e.value.status == -1
    with pytest.raises(moe.MoEError) as e:
        moe.W4Weights(torch.zeros((2, 64, 128), dtype=torch.bfloat16), torch.zeros((2, 128, 32), dtype=torch.bfloat16), group)
    assert e.value.status == -1
