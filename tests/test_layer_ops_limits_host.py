"""Norm, rotary positions, latent append and latent attention on the host: sizes and refusals at the ends of what their calls take.  No GPU:
no pointer is dereferenced."""
import pytest

from block_scaled_fp4_moe_gb300 import _build, attn
from test_layer_ops_host import ALIGN, INVALID, norm, rotary


@pytest.fixture(scope="module")
def L():
    _build.build()
    return attn.lib()


@pytest.mark.parametrize("heads", [1, 15, 16, 17, 64, 65, 96, 128, 129, 256])
@pytest.mark.parametrize("latent", [256, 512])
def test_latent_workspace_is_for_every_step_of_up_to_its_sizes(L, heads, latent):
    """It grows with T and with B, although a step's own units and parts do not."""
    size = attn.moe_latent_attention_workspace_size
    tokens = [*range(1, 41), 63, 64, 65, 127, 128, 129, 300, 1000, 5000, 1 << 20]
    requests = [*range(1, 41), 63, 64, 65, 152, 153, 256, 257, 1000, 8192]
    tokens = [t for t in tokens if t * heads < 1 << 31]
    sizes = {(t, b): size(t, b, heads, latent) for t in tokens for b in requests}
    assert min(sizes.values()) > 0
    for i, t in enumerate(tokens):
        for j, b in enumerate(requests):
            assert i == 0 or sizes[t, b] >= sizes[tokens[i - 1], b], (t, b)
            assert j == 0 or sizes[t, b] >= sizes[t, requests[j - 1]], (t, b)


SHARED = [(128, 128), (128, 256), (128, 504), (1024, 1024), (1 << 60, 1 << 60)]             # strides of tokens and heads, for 2 heads of 128 and more
SHARED_BY_8 = SHARED + [(256, 128), (1016, 128), (384, 256), (640, 384)]


def test_rotary_refuses_outputs_whose_rows_share_values(L):
    """4 tokens: a row of one of them that is, or reaches into, another's of another head."""
    for st, sh in SHARED_BY_8:
        assert rotary(L, qot=st, qoh=sh) == INVALID, (st, sh)
    for st, sh in SHARED:
        assert rotary(L, kot=st, koh=sh) == INVALID, (st, sh)


def test_norm_refuses_y_over_rows_of_x_that_lie_further_apart(L):
    for kw in (dict(ldx=520), dict(ldx=1024), dict(ldx=520, T=2), dict(ldx=1 << 40, res=0, res_out=0)):
        assert norm(L, **kw) == INVALID, kw
    assert norm(L, ldx=516) == ALIGN
