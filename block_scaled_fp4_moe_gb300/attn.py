"""Python binding of the attention half (include/moe_attn.h): the C-ABI calls
under the same names.

Argument marshalling only, as in ``moe``: tensors are passed as device
pointers, all of a call's on one device, the stream is torch's current stream of that device unless one is given, a nonzero
status raises ``moe.MoEError``, and the workspace is a uint8 CUDA tensor that is
zero-filled or passed through ``moe.moe_workspace_init`` once.  The tensors are checked (type, device,
layout, shape: ``ValueError``) in ``_attn_native.so`` (csrc/binding.cpp), which passes their addresses
on to the library that ``moe.lib()`` has loaded.

A serving step calls, per step, ``moe_kv_build_tables``, and per layer ``moe_rms_norm``,
``moe_linear_fp8`` (query, key and value heads), ``moe_rotary``, ``moe_kv_append``,
``moe_kv_attention``, ``moe_linear_fp8`` (output), ``moe_rms_norm`` with the residual sum and ``moe.moe_layer_forward``;
with one latent vector a token for all heads, ``moe_latent_append`` and ``moe_latent_attention`` in the places of
the other two.  ``examples/attention_step.py`` runs both.
"""
from __future__ import annotations

import ctypes as C
import importlib.util
import math
import os

import torch

from . import _build, moe


class _Cache(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("k_scale", C.c_void_p), ("v_scale", C.c_void_p),
                ("num_blocks", C.c_int32), ("kv_heads", C.c_int32), ("head_dim", C.c_int32), ("block_size", C.c_int32)]


class _LatentCache(C.Structure):
    _fields_ = [("data", C.c_void_p), ("num_blocks", C.c_int32), ("latent_dim", C.c_int32), ("block_size", C.c_int32)]


_p, _i, _l, _s, _f = C.c_void_p, C.c_int, C.c_int64, C.c_size_t, C.c_float
_SIG = {
    "moe_kv_build_tables": (_i, [_p, _p, _i, _i, _i, _p, _i, _p, _p, _i, _p, _p, _p, _p, _p, _p, _s, _p]),
    "moe_kv_append": (_i, [_p, _l, _l, _p, _l, _l, _p, _i, C.POINTER(_Cache), _p, _s, _p]),
    "moe_kv_attention_workspace_size": (_s, [_i, _i, _i, _i, _i]),
    "moe_kv_attention": (_i, [_p, _l, _l, _i, _i, C.POINTER(_Cache), _p, _i, _p, _p, _i, _f, _i, _i, _p, _p, _p, _s, _p]),
    "moe_quantize_fp8_weight": (_i, [_p, _i, _i, _p, _p, _p]),
    "moe_linear_fp8_workspace_size": (_s, [_i, _i, _i]),
    "moe_linear_fp8": (_i, [_p, _l, _i, _p, _p, _i, _i, _p, _p, _s, _p]),
    "moe_rms_norm": (_i, [_p, _l, _i, _i, _p, _p, _l, _f, _p, _p, _i, _p, _f, _p, _p]),
    "moe_rotary": (_i, [_p, _l, _l, _p, _l, _l, _i, _p, _l, _l, _p, _l, _l, _i, _i, _i, _p, _p, _i, _f, _i, _i, _p, _p, _f, _p]),
    "moe_latent_append": (_i, [_p, _l, _p, _l, _p, _i, _p, _p, _f, _i, _p, _f, C.POINTER(_LatentCache), _p, _s, _p]),
    "moe_latent_attention_workspace_size": (_s, [_i, _i, _i, _i]),
    "moe_latent_attention": (_i, [_p, _l, _l, _p, _l, _l, _i, _i, C.POINTER(_LatentCache), _p, _i, _p, _p, _i, _f, _i, _p, _p, _p, _s, _p]),
}
_ready: dict[int, C.CDLL] = {}


def lib() -> C.CDLL:
    """The library of ``moe.lib()`` with the signatures of moe_attn.h."""
    L = moe.lib()
    if id(L) not in _ready:
        for name, (res, args) in _SIG.items():
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _ready[id(L)] = L
    return L


def exported_symbols() -> list[str]:
    return list(_SIG)


_native_module = None
_bound = 0                          # address of the library that the module calls


def _native():
    """The compiled side of the calls, bound to the library in use."""
    global _native_module, _bound
    L = moe._libs.get(moe._debug) or moe.lib()
    if _bound != id(L):
        if _native_module is None:
            if not os.path.exists(_build.BINDING_PATH):
                raise RuntimeError(f"{_build.BINDING_PATH} is missing: run __graft_entry__.build() "
                                   "(or python -m block_scaled_fp4_moe_gb300._build)")
            spec = importlib.util.spec_from_file_location("_attn_native", _build.BINDING_PATH)
            _native_module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(_native_module)
        lib()
        _native_module.set_library(*[C.cast(getattr(L, name), C.c_void_p).value for name in
                                     ("moe_kv_build_tables", "moe_kv_append", "moe_kv_attention", "moe_quantize_fp8_weight",
                                      "moe_linear_fp8", "moe_rms_norm", "moe_rotary", "moe_latent_append", "moe_latent_attention")])
        _bound = id(L)
    return _native_module


def _stream(stream):
    """None (torch's current stream, found by the compiled side) or the stream's address."""
    return stream if stream is None else stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


class KVCache:
    """The paged E4M3 cache (codes and scale bytes as uint8 tensors):
    k [num_blocks, kv_heads, block_size/16, head_dim/16, 16 tokens, 16 dims],
    v [num_blocks, kv_heads, block_size/16, head_dim, 16 tokens],
    k_scale, v_scale [num_blocks, kv_heads]."""
    __slots__ = ("k", "v", "k_scale", "v_scale")

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor):
        _native().check_cache(k, v, k_scale, v_scale)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale

    @property
    def num_blocks(self) -> int:
        return self.k.shape[0]

    @property
    def kv_heads(self) -> int:
        return self.k.shape[1]

    @property
    def head_dim(self) -> int:
        return 16 * self.k.shape[3]

    @property
    def block_size(self) -> int:
        return 16 * self.k.shape[2]

    @staticmethod
    def empty(num_blocks: int, kv_heads: int, head_dim: int, block_size: int, device="cuda") -> "KVCache":
        """A cache whose blocks hold nothing yet (its memory is not cleared)."""
        def make(*shape):
            return torch.empty(shape, dtype=torch.uint8, device=device)
        subs = block_size // 16
        return KVCache(make(num_blocks, kv_heads, subs, head_dim // 16, 16, 16), make(num_blocks, kv_heads, subs, head_dim, 16),
                       make(num_blocks, kv_heads), make(num_blocks, kv_heads))


class FP8Weight:
    """codes uint8 [N, K] (E4M3) and scale uint8 [ceil(N/128), ceil(K/128)] (E8M0)."""
    __slots__ = ("codes", "scale")

    def __init__(self, codes: torch.Tensor, scale: torch.Tensor):
        _native().check_weight(codes, scale)
        self.codes, self.scale = codes, scale

    @property
    def n(self) -> int:
        return self.codes.shape[0]

    @property
    def k(self) -> int:
        return self.codes.shape[1]

    @staticmethod
    def from_dense(w: torch.Tensor, stream=None) -> "FP8Weight":
        """Quantises w bf16 [N, K] (moe_quantize_fp8_weight)."""
        n, k = w.shape
        out = FP8Weight(torch.empty((n, k), dtype=torch.uint8, device=w.device),
                        torch.empty((-(-n // 128), -(-k // 128)), dtype=torch.uint8, device=w.device))
        moe_quantize_fp8_weight(w, out, stream)
        return out


class LatentCache:
    """The paged cache of latent vectors: data bf16 [num_blocks, block_size, latent_dim + 64], a token's latent vector and
    rotary key side by side."""
    __slots__ = ("data",)

    def __init__(self, data: torch.Tensor):
        _native().check_latent_cache(data)
        self.data = data

    @property
    def num_blocks(self) -> int:
        return self.data.shape[0]

    @property
    def block_size(self) -> int:
        return self.data.shape[1]

    @property
    def latent_dim(self) -> int:
        return self.data.shape[2] - 64

    @staticmethod
    def empty(num_blocks: int, latent_dim: int, block_size: int, device="cuda") -> "LatentCache":
        """A cache whose blocks hold nothing yet (its memory is not cleared)."""
        return LatentCache(torch.empty((num_blocks, block_size, latent_dim + 64), dtype=torch.bfloat16, device=device))


class RotaryTable:
    """Frequencies of the rotated pairs: turns int64 [pairs], in units of 2^-64 turns a position (the bits of the unsigned
    number), and the factor of cosines and sines."""
    __slots__ = ("turns", "amplitude")

    def __init__(self, turns: torch.Tensor, amplitude: float = 1.0):
        self.turns, self.amplitude = turns, amplitude

    @staticmethod
    def make(dims: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0, original_len: int = 0, fast: float = 32.0,
             slow: float = 1.0, amplitude: float | None = None, device="cuda", ramp: str = "turns") -> "RotaryTable":
        """A table for ``dims`` rotated dims: pair i turns by base^(-2 i / dims) radians a position.  For contexts ``factor`` times
        as long as a model was trained on, ``scaling`` is "linear" (all frequencies divided by it), "base" (the base enlarged so that the
        slowest pair's is), or "parts" (pairs that turn ``fast`` times or more in ``original_len`` positions as they are, those that
        turn ``slow`` times or fewer divided; the amplitude is 0.1 ln(factor) + 1 unless one is given).  Between those a frequency
        is the average of both, its share of the one a straight line in ``ramp``: "turns", how often the pair turns, or "pairs", its
        index, from the last whole one at or before which a pair would turn ``fast`` times to the first at or after which ``slow`` times.  The
        two are up to four times apart in the middle: take the one that the weights were trained with."""
        if dims <= 0 or dims % 2 or not base > 0 or not (factor > 0 and math.isfinite(factor)):
            raise ValueError(f"dims {dims}, base {base}, factor {factor}: expected an even number and positive ones")
        if scaling not in (None, "linear", "base", "parts"):
            raise ValueError(f"scaling: expected linear, base or parts, got {scaling!r}")
        if scaling is None and factor != 1.0:
            raise ValueError("factor: expected with a scaling only")
        if scaling == "parts" and not (original_len > 0 and fast > slow >= 0):
            raise ValueError("scaling by parts: expected original_len > 0 and fast > slow >= 0")
        if ramp not in ("turns", "pairs"):
            raise ValueError(f"ramp: expected turns or pairs, got {ramp!r}")
        if ramp == "pairs":
            if scaling != "parts" or not (slow > 0 and base > 1):
                raise ValueError("ramp over pairs: expected scaling by parts, slow > 0 and a base above 1")
            first, last = (dims * math.log(original_len / (2 * math.pi * n)) / (2 * math.log(base)) for n in (fast, slow))
            first, last = max(math.floor(first), 0), min(math.ceil(last), dims - 1)
        if scaling == "base":
            if dims < 4:
                raise ValueError("scaling of the base: expected two pairs or more")
            base *= factor ** (dims / (dims - 2))
        turns = []
        for i in range(dims // 2):
            f = base ** (-2 * i / dims)
            if scaling == "linear":
                f /= factor
            elif scaling == "parts":
                keep = (original_len * f / (2 * math.pi) - slow) / (fast - slow) if ramp == "turns" else (last - i) / max(last - first, 1e-3)
                keep = min(max(keep, 0.0), 1.0)
                f = f * keep + f / factor * (1 - keep)
            whole = round(f / (2 * math.pi) * 2.0 ** 64) % (1 << 64)
            turns.append(whole - (1 << 64) if whole >> 63 else whole)
        if amplitude is None:
            amplitude = 0.1 * math.log(factor) + 1 if scaling == "parts" and factor > 1 else 1.0
        return RotaryTable(torch.tensor(turns, dtype=torch.int64, device=device), amplitude)


def alloc_workspace(max_tokens: int, max_requests: int, q_heads: int, cache: KVCache | LatentCache, weights=()) -> torch.Tensor:
    """A workspace for steps of up to these sizes: the attention's over this cache and, for
    ``weights`` (FP8Weight), the projections'."""
    latent = isinstance(cache, LatentCache)
    n = max([512, moe_latent_attention_workspace_size(max_tokens, max_requests, q_heads, cache.latent_dim) if latent else
             moe_kv_attention_workspace_size(max_tokens, max_requests, q_heads, cache.kv_heads, cache.head_dim)] +
            [moe_linear_fp8_workspace_size(max_tokens, *w.codes.shape) for w in weights])
    ws = torch.empty(n, dtype=torch.uint8, device=cache.data.device if latent else cache.k.device)
    with torch.cuda.device(ws.device):
        moe.moe_workspace_init(ws)
    return ws


def moe_kv_build_tables(ctx_lens, new_lens, block_size, free_blocks, free_head, block_table, kv_lens, q_offsets, slot_map,
                        positions, free_head_out, ws, stream=None):
    st = _native().kv_build_tables(ctx_lens, new_lens, block_size, free_blocks, free_head, block_table, kv_lens, q_offsets, slot_map,
                                   positions, free_head_out, ws, _stream(stream))
    if st:
        raise moe.MoEError(st, "moe_kv_build_tables")


def moe_kv_append(k, v, slot_map, cache: KVCache, ws, stream=None):
    """k, v bf16 [T, kv_heads, head_dim]; views with strides are taken as they are."""
    st = _native().kv_append(k, v, slot_map, cache.k, cache.v, cache.k_scale, cache.v_scale, ws, _stream(stream))
    if st:
        raise moe.MoEError(st, "moe_kv_append")


def moe_kv_attention_workspace_size(T: int, B: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    return int(lib().moe_kv_attention_workspace_size(T, B, q_heads, kv_heads, head_dim))


def moe_kv_attention(q, cache: KVCache, block_table, q_offsets, kv_lens, softmax_scale, out, lse, ws, causal=True, window=0,
                     stream=None):
    """q bf16 [T, q_heads, head_dim] (strided views are taken as they are), out
    bf16 of the same shape, contiguous; lse fp32 [T, q_heads] or None."""
    st = _native().kv_attention(q, cache.k, cache.v, cache.k_scale, cache.v_scale, block_table, q_offsets, kv_lens, softmax_scale, out,
                                lse, ws, causal, window, _stream(stream))
    if st:
        raise moe.MoEError(st, "moe_kv_attention")


def moe_quantize_fp8_weight(w, out: FP8Weight, stream=None):
    st = _native().quantize_fp8_weight(w, out.codes, out.scale, _stream(stream))
    if st:
        raise moe.MoEError(st, "moe_quantize_fp8_weight")


def moe_linear_fp8_workspace_size(T: int, N: int, K: int) -> int:
    return int(lib().moe_linear_fp8_workspace_size(T, N, K))


def moe_linear_fp8(x, w: FP8Weight, y, ws, stream=None):
    """y bf16 [T, N] = x W^T; x bf16 [T, K], rows may lie further apart than K."""
    st = _native().linear_fp8(x, w.codes, w.scale, y, ws, _stream(stream))
    if st:
        raise moe.MoEError(st, "moe_linear_fp8")


def moe_rms_norm(x, weight, eps, y, residual=None, residual_out=None, post_weight=None, gate=None, scale=1.0, stream=None):
    """x bf16 [T, H], rows may lie further apart than H; residual and residual_out bf16 or fp32 [T, H]; gate bf16 [H] or [T, H];
    weight and y may be None where residual_out is given."""
    st = _native().rms_norm(x, weight, eps, y, residual, residual_out, post_weight, gate, scale, _stream(stream))
    if st:
        raise moe.MoEError(st, "moe_rms_norm")


def moe_rotary(q, positions, table: RotaryTable, q_out, k=None, k_out=None, interleaved=False, offset=0, q_norm=None, k_norm=None,
               eps=1e-6, stream=None):
    """q, k bf16 [T, heads, head_dim] (strided views are taken as they are); q_out and k_out may be q and k."""
    st = _native().rotary(q, positions, table.turns, table.amplitude, q_out, k, k_out, interleaved, offset, q_norm, k_norm, eps,
                          _stream(stream))
    if st:
        raise moe.MoEError(st, "moe_rotary")


def moe_latent_append(c, k, slot_map, cache: LatentCache, ws, positions=None, table: RotaryTable | None = None, interleaved=False,
                      norm=None, eps=1e-6, stream=None):
    """c bf16 [T, latent_dim] and k bf16 [T, 64], rows may lie further apart; k is rotated where positions and a table are given (tokens
    whose position is negative are left out then), c normed where norm is."""
    turns, amplitude = (None, 1.0) if table is None else (table.turns, table.amplitude)
    st = _native().latent_append(c, k, slot_map, cache.data, ws, positions, turns, amplitude, interleaved, norm, eps, _stream(stream))
    if st:
        raise moe.MoEError(st, "moe_latent_append")


def moe_latent_attention_workspace_size(T: int, B: int, heads: int, latent_dim: int) -> int:
    return int(lib().moe_latent_attention_workspace_size(T, B, heads, latent_dim))


def moe_latent_attention(q_latent, q_rope, cache: LatentCache, block_table, q_offsets, kv_lens, softmax_scale, out, lse, ws, causal=True,
                         stream=None):
    """q_latent bf16 [T, heads, latent_dim] and q_rope bf16 [T, heads, 64] (strided views are taken as they are), out bf16
    [T, heads, latent_dim], contiguous; lse fp32 [T, heads] or None."""
    st = _native().latent_attention(q_latent, q_rope, cache.data, block_table, q_offsets, kv_lens, softmax_scale, out, lse, ws, causal,
                                    _stream(stream))
    if st:
        raise moe.MoEError(st, "moe_latent_attention")
