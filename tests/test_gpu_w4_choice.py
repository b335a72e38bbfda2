"""Which kernels a decode batch through 4-bit experts takes where a token has more
routes than there are experts: two launches token by token, four with the routes
grouped by expert."""
import pytest
import torch

import mixture_experts_routing_gb300 as moe
from test_gpu_w4 import DEV, Batch, gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,h,i,group,launches", [
    (31, 2048, 768, 64, 4), (30, 2048, 768, 64, 4),  # 150 MB of weights would be read again
    (16, 64, 64, 32, 2), (15, 64, 64, 32, 2),        # 0.2 MB
])
def test_more_routes_than_experts(n, h, i, group, launches):
    e, k = 2, 16
    b = Batch(n, h, e, e, i, group)
    g = gen(n)
    b.k, b.cfg = k, moe.W4Config(n, h, e, k, i, group)
    b.ids = torch.randint(0, e, (n, k), device=DEV, generator=g, dtype=torch.int32)
    b.p = torch.softmax(torch.randn((n, k), device=DEV, generator=g), 1)
    b.ws = moe.alloc_w4_workspace(b.cfg, DEV)
    before = moe.launch_count()
    b.run()
    assert moe.launch_count() - before == launches
    b.check()
