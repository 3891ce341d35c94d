"""What the latent attention's weights in bf16 leave of its outputs: the same rounded weights make the products and the sum that they are
divided by, so that a row's output is an average of its tokens' values, whatever the weights' roundings."""
import pytest
import torch

import layer_ops_reference as ref
from block_scaled_fp4_moe_gb300 import _build, moe
from test_gpu_layer_ops import Step, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


@pytest.mark.parametrize("kv,n,heads,latent,block", [([200], [1], 16, 512, 64), ([200, 300], [1, 1], 96, 256, 16), ([20000], [1], 64, 512, 64),
                                                     ([9000], [2], 40, 256, 128), ([700], [20], 16, 512, 32)])
def test_a_row_that_one_token_dominates_is_that_token(kv, n, heads, latent, block):
    """Weights 2^28 to 2^31.3 times the others', below the 2^32 at which references move: others have less than 20000 / 2^28 = 2^-13.7 of the
    sum, and values of magnitude 1 to 2 that one token has to itself are away from the next bf16 by 2^-9 at least (2^-8 from 1 up)."""
    s = Step(kv, n, heads, latent, block, seed=60)
    s.scale = 0.6931
    s.ql, s.qr = torch.zeros_like(s.ql), torch.zeros_like(s.qr)
    s.qr[..., 0] = (1 + torch.arange(heads, device="cuda") % 16 / 128).to(torch.bfloat16)
    s.data[..., latent] = 0.0
    value = (1 + torch.arange(latent, device="cuda") % 128 / 128).to(torch.bfloat16) * (1 - 2 * (torch.arange(latent, device="cuda") % 3 == 0).to(torch.bfloat16))
    for b, k in enumerate(kv):
        page, off = s.slot(b, k * 5 // 8 + 5)              # not the first of a tile
        s.data[page, off, :latent] = value
        s.data[page, off, latent] = 28.0
    out, lse = s.run()
    assert moe.moe_check_device_status(s.ws) == 0
    assert torch.equal(out, value.expand_as(out)), f"{(out != value).sum().item()} of {out.numel()} values are another's"
    want = s.scale * 28.0 * s.qr[..., 0].double()          # log(1 + 2^-13.7) is below 2^-13.6
    assert ((lse.double() - want).abs() <= 2.0 ** -13.6 + 4 * ref.U32 * want).all()


@pytest.mark.parametrize("kv,n,heads,latent", [([1000, 70], [1, 2], 16, 512), ([15000], [1], 64, 256), ([900, 300], [1, 1], 128, 512)])
@pytest.mark.parametrize("spread", [1.0, 3.0, 6.0])
def test_outputs_are_averages_of_the_values(kv, n, heads, latent, spread):
    """Weights p (1 + e) with |e| <= 2^-8 over their sum: out - o = sum p e (c - o) / (1 + sum p e), so that what a token's rounding moves is its
    distance from the output, not its value.  Scores with this standard deviation."""
    s = Step(kv, n, heads, latent, 64, seed=61)
    s.scale = spread * (latent + 64) ** -0.5
    out, lse = s.run()
    assert moe.moe_check_device_status(s.ws) == 0
    # fp32's share, and lse
    _, _, want_lse, lse_bound = ref.latent_attention(s.ql, s.qr, s.data, s.table, s.offsets, s.kv, s.scale)
    within(lse, want_lse, lse_bound, "lse")
    q = torch.cat((s.ql, s.qr), -1).double()
    for b, k in enumerate(kv):
        keys = s.data[s.table[b, : -(-k // 64)].long()].double().reshape(-1, latent + 64)[:k]
        for t in range(s.offsets[b], s.offsets[b + 1]):
            seen = k - (s.offsets[b + 1] - t) + 1
            c = keys[:seen, :latent]
            x = s.scale * (q[t] @ keys[:seen].T)
            p = torch.softmax(x, -1)
            o = p @ c
            away = torch.stack([(p[h, :, None] * (c - o[h]).abs()).sum(0) for h in range(heads)])
            delta = (s.scale * (latent + 64) * ref.U32 * (q[t].abs() @ keys[:seen].abs().T)).amax(-1) + 4 * ref.U32 * x.abs().amax(-1)
            loss = (2 * torch.expm1(2 * delta) + (16 + 2 * seen) * ref.U32)[:, None] * (p @ c.abs())
            before = ref.U16 / (1 - ref.U16) * away + 1.01 * loss
            within(out[t], o, before + ref.U16 * (o.abs() + before) + 1e-38, f"token {t}")
