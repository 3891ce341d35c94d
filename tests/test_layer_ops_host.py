"""Norm, rotary positions, latent append and latent attention on the host: bad arguments are refused before a GPU is touched, and the
tables of frequencies are the formulas'.  No GPU: no pointer is dereferenced."""
import ctypes as C
import math

import pytest

from block_scaled_fp4_moe_gb300 import _build, attn, moe

FAKE = 1 << 40
OK, INVALID, SHAPE, ALIGN, SMALL = (moe.MOE_OK, moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED_SHAPE, moe.MOE_ERR_MISALIGNED,
                                    moe.MOE_ERR_WORKSPACE_TOO_SMALL)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    _build.build()
    return attn.lib()


def p(x=FAKE):
    return C.c_void_p(x)


def norm(L, x=FAKE, ldx=512, T=4, H=512, post=0, gate=0, ldg=0, scale=1.0, res=FAKE, res_out=FAKE, wide=0, weight=FAKE, eps=1e-6, y=FAKE):
    return L.moe_rms_norm(p(x), ldx, T, H, p(post), p(gate), ldg, scale, p(res), p(res_out), wide, p(weight), eps, p(y), None)


def test_norm_refusals(L):
    for kw in (dict(T=-1), dict(H=0), dict(H=-8), dict(eps=-1e-6), dict(eps=NAN), dict(eps=INF), dict(scale=NAN), dict(scale=INF), dict(wide=2), dict(x=0),
               dict(y=0), dict(weight=0), dict(y=0, weight=0, res_out=0), dict(ldx=504), dict(gate=FAKE, ldg=8), dict(gate=FAKE, ldg=-512)):
        assert norm(L, **kw) == INVALID, kw
    for kw in (dict(H=508, ldx=512), dict(H=32776, ldx=32776), dict(T=(1 << 20) + 1)):
        assert norm(L, **kw) == SHAPE, kw
    for kw in (dict(x=FAKE + 8), dict(y=FAKE + 2), dict(res=FAKE + 4), dict(res_out=FAKE + 8), dict(weight=FAKE + 8), dict(post=FAKE + 2), dict(gate=FAKE + 8),
               dict(ldx=516), dict(gate=FAKE, ldg=516)):
        assert norm(L, **kw) == ALIGN, kw
    assert norm(L, T=0, x=0) == OK


def rotary(L, q=FAKE, qt=1024, qh=128, qo=FAKE + 4096, qot=1024, qoh=128, hq=8, k=FAKE, kt=1024, kh=128, ko=FAKE + 4096, kot=1024, koh=128, hk=2, T=4, D=128,
           pos=FAKE, turns=FAKE, pairs=64, amp=1.0, inter=0, offset=0, qn=0, kn=0, eps=1e-6):
    return L.moe_rotary(p(q), qt, qh, p(qo), qot, qoh, hq, p(k), kt, kh, p(ko), kot, koh, hk, T, D, p(pos), p(turns), pairs, amp, inter, offset, p(qn), p(kn),
                        eps, None)


def test_rotary_refusals(L):
    for kw in (dict(T=-1), dict(hq=0), dict(hk=-1), dict(D=0), dict(pairs=0), dict(offset=-8), dict(amp=NAN), dict(amp=INF), dict(eps=-1.0), dict(inter=2),
               dict(qt=-8), dict(koh=-8), dict(q=0), dict(qo=0), dict(k=0), dict(ko=0), dict(pos=0), dict(turns=0), dict(qo=FAKE, qot=2048),
               dict(ko=FAKE, koh=256), dict(qoh=0), dict(qot=0), dict(koh=64), dict(kot=120)):
        assert rotary(L, **kw) == INVALID, kw
    for kw in (dict(T=(1 << 20) + 1), dict(hq=1025), dict(hk=1025), dict(D=264), dict(D=132), dict(pairs=4), dict(pairs=60), dict(offset=8), dict(pairs=72),
               dict(offset=4, pairs=56), dict(pairs=1 << 30)):
        assert rotary(L, **kw) == SHAPE, kw
    for kw in (dict(q=FAKE + 8), dict(qo=FAKE + 2), dict(k=FAKE + 8), dict(ko=FAKE + 4), dict(pos=FAKE + 2), dict(turns=FAKE + 4), dict(qn=FAKE + 8),
               dict(kn=FAKE + 2), dict(qt=1028), dict(qoh=132), dict(kt=1020)):
        assert rotary(L, **kw) == ALIGN, kw
    assert rotary(L, T=0, q=0) == OK
    assert rotary(L, hk=0, k=0, ko=0, kt=1, T=0) == OK                   # without k its arguments are not looked at


def cache(data=FAKE, nb=4, dim=512, bs=64):
    return C.byref(attn._LatentCache(data, nb, dim, bs))


BAD_CACHES = [(dict(data=0), INVALID), (dict(nb=0), INVALID), (dict(nb=-1), INVALID), (dict(dim=0), SHAPE), (dict(dim=128), SHAPE), (dict(dim=576), SHAPE),
              (dict(bs=48), SHAPE), (dict(bs=8), SHAPE), (dict(nb=1 << 25), SHAPE), (dict(data=FAKE + 8), ALIGN)]


def append(L, c=FAKE, ldc=576, k=FAKE, ldk=576, slots=FAKE, T=3, pos=FAKE, turns=FAKE, amp=1.0, inter=0, w=FAKE, eps=1e-6, to=None, ws=FAKE, wsb=1 << 20):
    return L.moe_latent_append(p(c), ldc, p(k), ldk, p(slots), T, p(pos), p(turns), amp, inter, p(w), eps, to or cache(), p(ws), wsb, None)


def test_latent_append_refusals(L):
    for kw, want in BAD_CACHES:
        assert append(L, to=cache(**kw)) == want, kw
    assert L.moe_latent_append(p(), 576, p(), 576, p(), 1, None, None, 1.0, 0, None, 0.0, None, p(), 1 << 20, None) == INVALID
    for kw in (dict(T=-1), dict(ldc=-8), dict(ldk=-8), dict(pos=0), dict(turns=0), dict(amp=NAN), dict(inter=3), dict(eps=NAN), dict(c=0), dict(k=0),
               dict(slots=0), dict(ws=0)):
        assert append(L, **kw) == INVALID, kw
    for kw in (dict(c=FAKE + 8), dict(k=FAKE + 2), dict(slots=FAKE + 4), dict(pos=FAKE + 1), dict(turns=FAKE + 4), dict(w=FAKE + 8), dict(ldc=580),
               dict(ldk=4), dict(ws=FAKE + 128)):
        assert append(L, **kw) == ALIGN, kw
    assert append(L, T=(1 << 24) + 1) == SHAPE
    assert append(L, wsb=511) == SMALL
    assert append(L, T=0, c=0) == OK


def attend(L, to=None, ql=FAKE, lt=8192, lh=512, qr=FAKE, rt=1024, rh=64, T=4, heads=16, table=FAKE, mb=8, qo=FAKE, kv=FAKE, B=2, scale=0.1, causal=1,
           out=FAKE, lse=FAKE, ws=FAKE, wsb=1 << 40):
    return L.moe_latent_attention(p(ql), lt, lh, p(qr), rt, rh, T, heads, to or cache(), p(table), mb, p(qo), p(kv), B, scale, causal, p(out), p(lse), p(ws),
                                  wsb, None)


def test_latent_attention_refusals(L):
    for kw, want in BAD_CACHES:
        assert attend(L, cache(**kw)) == want, kw
    for kw in (dict(T=-1), dict(B=-1), dict(heads=0), dict(mb=-1), dict(causal=2), dict(lt=-8), dict(lh=-8), dict(rt=-8), dict(rh=-8), dict(scale=NAN),
               dict(scale=INF), dict(scale=-1.0), dict(ql=0), dict(qr=0), dict(out=0), dict(qo=0), dict(kv=0), dict(table=0), dict(ws=0)):
        assert attend(L, **kw) == INVALID, kw
    for kw in (dict(T=(1 << 20) + 1), dict(B=8193), dict(heads=257), dict(mb=1 << 26)):
        assert attend(L, **kw) == SHAPE, kw
    for kw in (dict(ql=FAKE + 8), dict(qr=FAKE + 2), dict(out=FAKE + 8), dict(lse=FAKE + 2), dict(lt=8196), dict(lh=4), dict(rt=1020), dict(rh=2),
               dict(ws=FAKE + 64)):
        assert attend(L, **kw) == ALIGN, kw
    size = attn.moe_latent_attention_workspace_size
    need = size(4, 2, 16, 512)
    assert need > 0 and attend(L, wsb=need - 1) == SMALL
    assert attend(L, T=0, ql=0) == OK and attend(L, B=0) == OK
    assert size(4, 2, 0, 512) == size(4, 2, 257, 512) == size(4, 2, 16, 384) == size(-1, 2, 16, 512) == 0


def test_tables_are_the_formulas():
    """turns[i] / 2^64 = base^(-2 i / dims) / 2 pi, a frequency in turns; scaled ones against the scaling's definition."""
    def frequencies(*args, **kw):
        t = attn.RotaryTable.make(*args, device="cpu", **kw)
        return [(v % (1 << 64)) / 2.0 ** 64 * 2 * math.pi for v in t.turns.tolist()], t.amplitude
    plain = [10000.0 ** (-2 * i / 64) for i in range(32)]
    f, amp = frequencies(64)
    assert amp == 1.0 and len(f) == 32
    for a, b in zip(f, plain):
        assert abs(a - b) <= 1e-14 * b + 2.0 ** -62
    f, _ = frequencies(64, scaling="linear", factor=4.0)
    assert all(abs(a - b / 4) <= 1e-14 * b + 2.0 ** -62 for a, b in zip(f, plain))
    f, _ = frequencies(64, scaling="base", factor=8.0)
    assert abs(f[0] - 1) < 1e-14 and abs(f[-1] - plain[-1] / 8) < 1e-12 * plain[-1]
    f, amp = frequencies(64, scaling="parts", factor=40.0, original_len=4096)
    assert abs(amp - (0.1 * math.log(40) + 1)) < 1e-15
    for a, b in zip(f, plain):
        n = 4096 * b / (2 * math.pi)                       # turns in the trained context
        if n >= 32:
            assert abs(a - b) <= 1e-14 * b
        elif n <= 1:
            assert abs(a - b / 40) <= 1e-14 * b + 2.0 ** -62
        else:
            assert b / 40 < a < b
    assert frequencies(64, scaling="parts", factor=40.0, original_len=4096, amplitude=1.0)[1] == 1.0
    one = attn.RotaryTable.make(16, base=1.0, device="cpu")              # frequency 1 throughout: 1 / 2 pi turns
    assert all(abs((v % (1 << 64)) / 2.0 ** 64 - 1 / (2 * math.pi)) < 1e-16 for v in one.turns.tolist())


@pytest.mark.parametrize("kw", [dict(dims=0), dict(dims=7), dict(dims=64, base=0.0), dict(dims=64, factor=0.0), dict(dims=64, factor=INF), dict(dims=64, scaling="ntk"),
                                dict(dims=64, factor=2.0), dict(dims=64, scaling="parts", factor=2.0), dict(dims=2, scaling="base", factor=2.0),
                                dict(dims=64, scaling="parts", factor=2.0, original_len=10, fast=1.0, slow=2.0)])
def test_tables_that_make_no_sense_are_refused(kw):
    with pytest.raises(ValueError):
        attn.RotaryTable.make(device="cpu", **kw)


def test_binding_checks_shapes_types_and_devices(L):
    """The compiled checks name the tensor (stand-ins without memory: nothing is launched)."""
    torch = pytest.importorskip("torch")
    fake = pytest.importorskip("torch._subclasses.fake_tensor")
    if torch.cuda.is_available():
        pytest.skip("stand-ins for a second device need a machine without the first")
    with pytest.raises(ValueError, match="cache: expected a CUDA tensor"):
        attn.LatentCache(torch.zeros(1, 16, 576, dtype=torch.bfloat16))
    with fake.FakeTensorMode():
        def make(dtype, *shape, device="cuda:0"):
            return torch.empty(shape, dtype=dtype, device=device)

        def bf(*shape, **kw):
            return make(torch.bfloat16, *shape, **kw)
        f32, i32, i64, u8 = torch.float32, torch.int32, torch.int64, torch.uint8
        x, w = bf(4, 64), bf(64)
        calls = [
            ("x: expected a matrix", lambda: attn.moe_rms_norm(bf(64), w, 0.0, x)),
            ("x: expected BFloat16", lambda: attn.moe_rms_norm(make(f32, 4, 64), w, 0.0, x)),
            ("weight: expected shape", lambda: attn.moe_rms_norm(x, bf(32), 0.0, bf(4, 64))),
            ("y: expected shape", lambda: attn.moe_rms_norm(x, w, 0.0, bf(3, 64))),
            ("residual: expected BFloat16", lambda: attn.moe_rms_norm(x, w, 0.0, x, residual=make(torch.float16, 4, 64))),
            ("residual_out: expected BFloat16", lambda: attn.moe_rms_norm(x, w, 0.0, x, residual=x, residual_out=make(f32, 4, 64))),
            ("residual_out: expected Float", lambda: attn.moe_rms_norm(x, w, 0.0, x, residual=make(f32, 4, 64), residual_out=x)),
            ("gate: expected shape", lambda: attn.moe_rms_norm(x, w, 0.0, x, gate=bf(3, 64))),
            ("post_weight: expected a tensor on cuda:0 as x", lambda: attn.moe_rms_norm(x, w, 0.0, x, post_weight=bf(64, device="cuda:1"))),
        ]
        table = attn.RotaryTable(make(i64, 32))
        q, pos = bf(4, 2, 64), make(i32, 4)
        calls += [
            ("q: expected \\[tokens", lambda: attn.moe_rotary(bf(4, 64), pos, table, q)),
            ("q_out: expected shape", lambda: attn.moe_rotary(q, pos, table, bf(4, 1, 64))),
            ("positions: expected shape", lambda: attn.moe_rotary(q, make(i32, 5), table, q)),
            ("positions: expected Int", lambda: attn.moe_rotary(q, make(i64, 4), table, q)),
            ("turns: expected Long", lambda: attn.moe_rotary(q, pos, attn.RotaryTable(make(i32, 32)), q)),
            ("k_out: expected with k", lambda: attn.moe_rotary(q, pos, table, q, k=q)),
            ("k_norm: expected with k", lambda: attn.moe_rotary(q, pos, table, q, k_norm=w)),
            ("k: expected a tensor on cuda:0 as q", lambda: attn.moe_rotary(q, pos, table, q, k=bf(4, 2, 64, device="cuda:1"), k_out=q)),
        ]
        with pytest.raises(ValueError, match="cache: expected \\[blocks"):
            attn.LatentCache(bf(4, 16, 64))
        cache, slots, ws = attn.LatentCache(bf(4, 16, 320)), make(i64, 3), make(u8, 512)
        c, k = bf(3, 256), bf(3, 64)
        calls += [
            ("c: expected shape", lambda: attn.moe_latent_append(bf(3, 512), k, slots, cache, ws)),
            ("k: expected shape", lambda: attn.moe_latent_append(c, bf(3, 32), slots, cache, ws)),
            ("positions: expected with a table", lambda: attn.moe_latent_append(c, k, slots, cache, ws, positions=make(i32, 3))),
            ("turns: expected shape", lambda: attn.moe_latent_append(c, k, slots, cache, ws, make(i32, 3), attn.RotaryTable(make(i64, 16)))),
            ("norm: expected shape", lambda: attn.moe_latent_append(c, k, slots, cache, ws, norm=bf(64))),
            ("slot_map: expected a tensor on cuda:0", lambda: attn.moe_latent_append(c, k, make(i64, 3, device="cuda:1"), cache, ws)),
        ]
        ql, qr, one = bf(3, 4, 256), bf(3, 4, 64), make(i32, 1)
        rest = (one.view(1, 1), make(i32, 2), one, 1.0)
        calls += [
            ("q_latent: expected shape", lambda: attn.moe_latent_attention(bf(3, 4, 512), qr, cache, *rest, ql, None, ws)),
            ("q_rope: expected shape", lambda: attn.moe_latent_attention(ql, bf(3, 2, 64), cache, *rest, ql, None, ws)),
            ("out: expected shape", lambda: attn.moe_latent_attention(ql, qr, cache, *rest, bf(3, 4, 64), None, ws)),
            ("lse: expected shape", lambda: attn.moe_latent_attention(ql, qr, cache, *rest, ql, make(f32, 3), ws)),
            ("block_table: expected 1 rows", lambda: attn.moe_latent_attention(ql, qr, cache, make(i32, 2, 1), *rest[1:], ql, None, ws)),
            ("kv_lens: expected a tensor on cuda:0", lambda: attn.moe_latent_attention(ql, qr, cache, rest[0], rest[1], make(i32, 1, device="cuda:1"), 1.0, ql,
                                                                                   None, ws)),
        ]
        for match, call in calls:
            with pytest.raises(ValueError, match=match):
                call()
