"""Norm, rotary positions, latent append and latent attention at the ends of what their calls take."""
import pytest
import torch

from block_scaled_fp4_moe_gb300 import _build, attn, moe
from test_gpu_layer_ops import Step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


@pytest.mark.parametrize("heads,latent", [(16, 512), (96, 256), (5, 512)])
def test_a_workspace_for_many_requests_serves_steps_of_fewer(heads, latent):
    """More tokens than requests, in a workspace made for as many of either: that step's units are others, and its parts larger."""
    cache = attn.LatentCache.empty(1, latent, 64)
    ws = attn.alloc_workspace(64, 64, heads, cache)
    for kv, n in (([5000] * 4, [3, 1, 4, 2]), ([700] * 62, [2] + [1] * 61), ([9000], [2]), ([300] * 64, [1] * 64), ([20000], [64])):
        s = Step(kv, n, heads, latent, 64, seed=75)
        out, lse = s.run(ws=ws)
        want, want_lse = s.run()
        assert moe.moe_check_device_status(ws) == 0
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
