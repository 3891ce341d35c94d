"""Norm, rotary positions, latent append and latent attention on the host: sizes and refusals at the ends of what their calls take.  No GPU:
no pointer is dereferenced."""
import math

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


def frequencies(*args, **kw):
    return [(v % (1 << 64)) / 2.0 ** 64 * 2 * math.pi for v in attn.RotaryTable.make(*args, device="cpu", **kw).turns.tolist()]


@pytest.mark.parametrize("dims,base,factor,length,first,last", [(64, 10000.0, 40.0, 4096, 10, 23), (128, 1e6, 4.0, 32768, 23, 40), (64, 10000.0, 2.0, 16, 0, 4)])
def test_tables_scaled_by_parts_over_the_index_of_the_pair(dims, base, factor, length, first, last):
    """first, last: where base^(-2 i / dims) length / 2 pi is 32 and 1, rounded outwards (to 0 at least)."""
    turns = [length * base ** (-2 * i / dims) / (2 * math.pi) for i in range(dims // 2)]
    assert (first == 0 and turns[0] < 32) or turns[first] >= 32 > turns[first + 1]
    assert turns[last] <= 1 < turns[last - 1]
    got = frequencies(dims, base=base, scaling="parts", factor=factor, original_len=length, ramp="pairs")
    for i, f in enumerate(got):
        plain = base ** (-2 * i / dims)
        keep = 1.0 if i <= first else 0.0 if i >= last else 1 - (i - first) / (last - first)
        want = keep * plain + (1 - keep) * plain / factor
        assert abs(f - want) <= 1e-13 * plain + 2.0 ** -62, i


def test_tables_scaled_by_parts_over_the_turns():
    """The ramp that is meant where none is given: a share of (turns - 1) / 31 of the plain frequency, in the middle far from the other."""
    args = dict(scaling="parts", factor=40.0, original_len=4096)
    got, same, other = frequencies(64, **args), frequencies(64, ramp="turns", **args), frequencies(64, ramp="pairs", **args)
    assert got == same
    for i, f in enumerate(got):
        plain = 10000.0 ** (-2 * i / 64)
        keep = min(max((4096 * plain / (2 * math.pi) - 1) / 31, 0.0), 1.0)
        assert abs(f - (keep * plain + (1 - keep) * plain / 40)) <= 1e-13 * plain + 2.0 ** -62, i
    assert 4.2 < other[20] / got[20] < 4.4
    assert all(f == g for i, (f, g) in enumerate(zip(got, other)) if not 10 < i < 23)


@pytest.mark.parametrize("kw", [dict(ramp="index", scaling="parts"), dict(ramp="pairs"), dict(ramp="pairs", scaling="linear"), dict(ramp="pairs", scaling="parts", slow=0.0),
                                dict(ramp="pairs", scaling="parts", base=1.0)])
def test_ramps_that_make_no_sense_are_refused(kw):
    with pytest.raises(ValueError):
        attn.RotaryTable.make(64, factor=2.0 if "scaling" in kw else 1.0, original_len=4096, device="cpu", **kw)
