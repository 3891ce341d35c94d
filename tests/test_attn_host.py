"""The attention half's C ABI on the host: every function of moe_attn.h is
exported and bad arguments are refused before a GPU is touched; and the
tests' reference checked on its own (its format against the OCP table's anchors and
by brute force).  No GPU: no pointer is dereferenced."""
import ctypes as C
import os
import re

import numpy as np
import pytest

import attn_reference as ref
from block_scaled_fp4_moe_gb300 import _build, attn, moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 40
OK, INVALID, SHAPE, ALIGN, SMALL = (moe.MOE_OK, moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED_SHAPE, moe.MOE_ERR_MISALIGNED,
                                    moe.MOE_ERR_WORKSPACE_TOO_SMALL)


@pytest.fixture(scope="module")
def L():
    _build.build()
    return attn.lib()


def p(x=FAKE):
    return C.c_void_p(x)


def test_every_declared_function_is_exported(L):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "moe_attn.h")).read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", text)))
    assert declared == sorted(attn.exported_symbols())
    for name in declared:
        assert hasattr(L, name), name


def tables(L, ctx=FAKE, new=FAKE, B=2, T=4, bs=64, free=FAKE, nf=8, head=FAKE, table=FAKE, mb=4, kv=FAKE, qo=FAKE, slots=FAKE,
           pos=FAKE, out=FAKE + 256, ws=FAKE, wsb=1 << 20):
    return L.moe_kv_build_tables(p(ctx), p(new), B, T, bs, p(free), nf, p(head), p(table), mb, p(kv), p(qo), p(slots), p(pos), p(out),
                                 p(ws), wsb, None)


def test_build_tables_refusals(L):
    for kw in (dict(B=-1), dict(T=-1), dict(nf=-1), dict(mb=-1), dict(head=0), dict(qo=0), dict(out=0), dict(out=FAKE), dict(ctx=0),
               dict(new=0), dict(kv=0), dict(table=0), dict(slots=0), dict(pos=0), dict(free=0), dict(ws=0)):
        assert tables(L, **kw) == INVALID, kw
    for kw in (dict(bs=48), dict(bs=8), dict(bs=256), dict(B=8193), dict(T=(1 << 24) + 1), dict(mb=1 << 26)):
        assert tables(L, **kw) == SHAPE, kw
    for kw in (dict(ctx=FAKE + 2), dict(slots=FAKE + 4), dict(ws=FAKE + 16), dict(table=FAKE + 1)):
        assert tables(L, **kw) == ALIGN, kw
    assert tables(L, wsb=511) == SMALL


def cache(k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, nb=4, heads=8, dim=128, bs=64):
    return C.byref(attn._Cache(k, v, ks, vs, nb, heads, dim, bs))


BAD_CACHES = [(dict(k=0), INVALID), (dict(v=0), INVALID), (dict(ks=0), INVALID), (dict(vs=0), INVALID), (dict(nb=0), INVALID),
              (dict(heads=0), INVALID), (dict(dim=96), SHAPE), (dict(dim=0), SHAPE), (dict(bs=48), SHAPE), (dict(heads=1025), SHAPE),
              (dict(k=FAKE + 8), ALIGN), (dict(v=FAKE + 8), ALIGN)]


def append(L, c=None, k=FAKE, kt=1024, kh=128, v=FAKE, vt=1024, vh=128, slots=FAKE, T=3, ws=FAKE, wsb=1 << 20):
    return L.moe_kv_append(p(k), kt, kh, p(v), vt, vh, p(slots), T, c or cache(), p(ws), wsb, None)


def test_append_refusals(L):
    for kw, want in BAD_CACHES:
        assert append(L, cache(**kw)) == want, kw
    assert L.moe_kv_append(p(), 8, 8, p(), 8, 8, p(), 1, None, p(), 1 << 20, None) == INVALID
    for kw in (dict(T=-1), dict(kt=-8), dict(k=0), dict(v=0), dict(slots=0), dict(ws=0)):
        assert append(L, **kw) == INVALID, kw
    for kw in (dict(k=FAKE + 8), dict(v=FAKE + 2), dict(kt=1028), dict(vh=4), dict(slots=FAKE + 4), dict(ws=FAKE + 128)):
        assert append(L, **kw) == ALIGN, kw
    assert append(L, T=(1 << 24) + 1) == SHAPE
    assert append(L, wsb=100) == SMALL
    assert append(L, T=0, k=0) == OK                       # nothing to do


def attend(L, c=None, q=FAKE, qt=8192, qh=128, T=4, heads=64, table=FAKE, mb=8, qo=FAKE, kv=FAKE, B=2, scale=0.1, causal=1, window=0,
           out=FAKE, lse=FAKE, ws=FAKE, wsb=1 << 40):
    return L.moe_kv_attention(p(q), qt, qh, T, heads, c or cache(), p(table), mb, p(qo), p(kv), B, scale, causal, window, p(out), p(lse),
                              p(ws), wsb, None)


def test_attention_refusals(L):
    for kw, want in BAD_CACHES:
        assert attend(L, cache(**kw)) == want, kw
    for kw in (dict(T=-1), dict(B=-1), dict(heads=0), dict(heads=60), dict(mb=-1), dict(window=-1), dict(causal=2), dict(qt=-4),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=-1.0), dict(q=0), dict(out=0), dict(qo=0), dict(kv=0),
               dict(table=0), dict(ws=0)):
        assert attend(L, **kw) == INVALID, kw
    for kw in (dict(T=(1 << 20) + 1), dict(B=8193), dict(heads=8 * 257), dict(mb=1 << 26)):
        assert attend(L, **kw) == SHAPE, kw
    for kw in (dict(q=FAKE + 4), dict(out=FAKE + 2), dict(lse=FAKE + 2), dict(qt=8194), dict(qh=126), dict(ws=FAKE + 64)):
        assert attend(L, **kw) == ALIGN, kw
    need = attn.moe_kv_attention_workspace_size(4, 2, 64, 8, 128)
    assert need > 0 and attend(L, wsb=need - 1) == SMALL
    assert attend(L, T=0) == OK and attend(L, B=0) == OK
    assert attn.moe_kv_attention_workspace_size(4, 2, 60, 8, 128) == 0
    assert attn.moe_kv_attention_workspace_size(4, 2, 64, 8, 80) == 0


def linear(L, x=FAKE, ldx=512, T=4, codes=FAKE, scale=FAKE, N=256, K=512, y=FAKE, ws=FAKE, wsb=1 << 40):
    return L.moe_linear_fp8(p(x), ldx, T, p(codes), p(scale), N, K, p(y), p(ws), wsb, None)


def test_linear_refusals(L):
    for kw in (dict(T=-1), dict(N=0), dict(K=0), dict(x=0), dict(codes=0), dict(scale=0), dict(y=0), dict(ws=0), dict(ldx=504)):
        assert linear(L, **kw) == INVALID, kw
    for kw in (dict(K=520, ldx=520), dict(K=65552, ldx=65552), dict(N=(1 << 20) + 1), dict(T=(1 << 20) + 1)):
        assert linear(L, **kw) == SHAPE, kw
    for kw in (dict(x=FAKE + 8), dict(codes=FAKE + 8), dict(y=FAKE + 2), dict(ldx=516), dict(ws=FAKE + 8)):
        assert linear(L, **kw) == ALIGN, kw
    need = attn.moe_linear_fp8_workspace_size(4, 256, 512)
    assert need > 0 and linear(L, wsb=need - 1) == SMALL
    assert linear(L, T=0, x=0) == OK
    assert attn.moe_linear_fp8_workspace_size(4, 256, 520) == 0
    assert L.moe_quantize_fp8_weight(None, 4, 16, p(), p(), None) == INVALID
    assert L.moe_quantize_fp8_weight(p(), 4, 24, p(), p(), None) == SHAPE
    assert L.moe_quantize_fp8_weight(p(FAKE + 2), 4, 16, p(), p(), None) == ALIGN


def test_workspace_grows_with_the_sizes(L):
    size = attn.moe_linear_fp8_workspace_size
    assert 0 < size(1, 64, 128) <= size(4, 64, 4096) < size(4000, 64, 4096)
    assert attn.moe_kv_attention_workspace_size(1, 1, 8, 8, 64) < attn.moe_kv_attention_workspace_size(4096, 64, 128, 8, 128)


# ------------------------------------------------------- the reference itself

def test_reference_e4m3_anchors():
    path = os.path.join(ROOT, "tests", "golden", "e4m3_ocp_anchors.txt")
    seen = 0
    for line in open(path):
        part = line.split("#")[0].split()
        if len(part) >= 2:
            code, value = int(part[0], 0), float(part[1])
            assert np.isnan(value) and np.isnan(ref.TABLE[code]) or ref.TABLE[code] == value, line
            seen += 1
    assert seen > 0


def test_reference_rounding_by_brute_force():
    rng = np.random.default_rng(1)
    v = np.concatenate([rng.uniform(-448, 448, 500), rng.uniform(-0.05, 0.05, 500), ref.TABLE[:127],
                        (ref.TABLE[:126] + ref.TABLE[1:127]) / 2])     # ties too
    codes = ref.e4m3_codes(v)
    finite = [c for c in range(256) if not np.isnan(ref.TABLE[c])]
    for x, c in zip(v, codes):
        d = np.abs(ref.TABLE[finite] - x)
        best = [k for k, e in zip(finite, d) if e == d.min()]
        assert c in best
        if len({k & 0x7F for k in best}) > 1:
            assert c % 2 == 0
    assert ref.e4m3_codes(np.array([np.inf, np.nan, -np.inf])).tolist()[0] & 0x7F == 0x7F


def test_reference_exponent_is_the_least():
    for a in (1e-30, 0.3, 447.9, 448.0, 448.1, 896.0, 897.0, 3.3e38):
        e = ref.least_exponent(a)
        assert a <= 448 * 2.0 ** e and a > 448 * 2.0 ** (e - 1)
    assert ref.least_exponent(0.0) == -126 and ref.least_exponent(1e-45) == -126


def test_reference_cache_layout_round_trip():
    rng = np.random.default_rng(2)
    c = ref.Cache(3, 2, 64, 32)
    c.k[:], c.v[:] = rng.integers(0, 256, c.k.shape), rng.integers(0, 256, c.v.shape)
    k, v, ks, vs = c.layout()
    assert k.shape == (3, 2, 2, 4, 16, 16) and v.shape == (3, 2, 2, 64, 16)
    assert k[1, 0, 1, 2, 5, 7] == c.k[1, 0, 21, 39] and v[2, 1, 1, 40, 9] == c.v[2, 1, 25, 40]
    back = ref.Cache.from_layout(k, v, ks, vs)
    assert np.array_equal(back.k, c.k) and np.array_equal(back.v, c.v)


def test_binding_refuses_what_is_not_on_the_gpu(L):
    """The compiled checks name the tensor, before any address is passed on."""
    torch = pytest.importorskip("torch")
    u8 = torch.zeros(1, 1, 1, 4, 16, 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="k: expected a CUDA tensor"):
        attn.KVCache(u8, u8, u8, u8)
    with pytest.raises(ValueError, match="codes: expected a CUDA tensor"):
        attn.FP8Weight(torch.zeros(16, 16, dtype=torch.uint8), torch.zeros(1, 1, dtype=torch.uint8))
    with pytest.raises(ValueError, match="k: expected a tensor"):
        attn.KVCache(None, u8, u8, u8)
    i32 = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="ctx_lens"):
        attn.moe_kv_build_tables(i32, i32, 16, i32, i32, i32, i32, i32, i32, i32, i32, u8)
    with pytest.raises(ValueError, match="expected 6 arguments"):
        attn._native().linear_fp8(u8)


def test_binding_refuses_tensors_of_two_devices(L):
    """All of a call's tensors are on one device (stand-ins without memory: nothing is launched)."""
    torch = pytest.importorskip("torch")
    fake = pytest.importorskip("torch._subclasses.fake_tensor")
    if torch.cuda.is_available():
        pytest.skip("stand-ins for a second device need a machine without the first")
    with fake.FakeTensorMode():
        def u8(*shape, device="cuda:0"):
            return torch.empty(shape, dtype=torch.uint8, device=device)
        k, v, scale = (2, 1, 1, 4, 16, 16), (2, 1, 1, 64, 16), (2, 1)
        cache = attn.KVCache(u8(*k), u8(*v), u8(*scale), u8(*scale))
        for i in range(1, 4):
            parts = [u8(*shape, device="cuda:1" if j == i else "cuda:0") for j, shape in enumerate((k, v, scale, scale))]
            with pytest.raises(ValueError, match=f"{('k', 'v', 'k_scale', 'v_scale')[i]}: expected a tensor on cuda:0 as k, got cuda:1"):
                attn.KVCache(*parts)
        weight = attn.FP8Weight(u8(16, 16), u8(1, 1))
        with pytest.raises(ValueError, match="scale: expected a tensor on cuda:0 as codes"):
            attn.FP8Weight(u8(16, 16), u8(1, 1, device="cuda:1"))

        def bf16(*shape, device="cuda:0"):
            return torch.empty(shape, dtype=torch.bfloat16, device=device)
        i32 = [torch.empty(1, dtype=torch.int32, device=d) for d in ("cuda:0", "cuda:1")]
        i64 = [torch.empty(1, dtype=torch.int64, device=d) for d in ("cuda:0", "cuda:1")]
        calls = [("ws", lambda: attn.moe_linear_fp8(bf16(1, 16), weight, bf16(1, 16), u8(512, device="cuda:1"))),
                 ("y", lambda: attn.moe_linear_fp8(bf16(1, 16), weight, bf16(1, 16, device="cuda:1"), u8(512))),
                 ("codes", lambda: attn.moe_quantize_fp8_weight(bf16(16, 16, device="cuda:1"), weight)),
                 ("slot_map", lambda: attn.moe_kv_append(bf16(1, 1, 64), bf16(1, 1, 64), i64[1], cache, u8(512))),
                 ("q", lambda: attn.moe_kv_attention(bf16(1, 1, 64, device="cuda:1"), cache, i32[0].view(1, 1), i32[0], i32[0], 1.0, bf16(1, 1, 64),
                                                     None, u8(512))),
                 ("kv_lens", lambda: attn.moe_kv_attention(bf16(1, 1, 64), cache, i32[0].view(1, 1), i32[0], i32[1], 1.0, bf16(1, 1, 64), None,
                                                           u8(512))),
                 ("new_lens", lambda: attn.moe_kv_build_tables(i32[0], i32[1], 16, i32[0], i32[0], i32[0].view(1, 1), i32[0], i32[0], i64[0], i32[0],
                                                               i32[0], u8(512)))]
        for name, call in calls:
            with pytest.raises(ValueError, match=f"{name}: expected a tensor on cuda:"):
                call()
