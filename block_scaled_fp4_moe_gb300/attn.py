"""Python binding of the attention half (include/moe_attn.h): the C-ABI calls
under the same names.

Argument marshalling only, as in ``moe``: tensors are passed as device
pointers, the stream is torch's current stream unless one is given, a nonzero
status raises ``moe.MoEError``, and the workspace is a uint8 CUDA tensor that is
zero-filled or passed through ``moe.moe_workspace_init`` once.

A serving step calls, per step, ``moe_kv_build_tables``, and per layer
``moe_linear_fp8`` (query, key and value heads), ``moe_kv_append``,
``moe_kv_attention``, ``moe_linear_fp8`` (output) and ``moe.moe_layer_forward``;
``examples/attention_step.py`` runs one.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import moe
from .moe import _check


class _Cache(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("k_scale", C.c_void_p), ("v_scale", C.c_void_p),
                ("num_blocks", C.c_int32), ("kv_heads", C.c_int32), ("head_dim", C.c_int32), ("block_size", C.c_int32)]


_p, _i, _l, _s, _f = C.c_void_p, C.c_int, C.c_int64, C.c_size_t, C.c_float
_SIG = {
    "moe_kv_build_tables": (_i, [_p, _p, _i, _i, _i, _p, _i, _p, _p, _i, _p, _p, _p, _p, _p, _p, _s, _p]),
    "moe_kv_append": (_i, [_p, _l, _l, _p, _l, _l, _p, _i, C.POINTER(_Cache), _p, _s, _p]),
    "moe_kv_attention_workspace_size": (_s, [_i, _i, _i, _i, _i]),
    "moe_kv_attention": (_i, [_p, _l, _l, _i, _i, C.POINTER(_Cache), _p, _i, _p, _p, _i, _f, _i, _i, _p, _p, _p, _s, _p]),
    "moe_quantize_fp8_weight": (_i, [_p, _i, _i, _p, _p, _p]),
    "moe_linear_fp8_workspace_size": (_s, [_i, _i, _i]),
    "moe_linear_fp8": (_i, [_p, _l, _i, _p, _p, _i, _i, _p, _p, _s, _p]),
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


# A call's time on the host is that of its checks: these do one attribute each on the way through, and say what is wrong
# only when something is.  Addresses and the stream are passed as plain integers.

_bf16, _i32, _i64, _u8, _f32 = torch.bfloat16, torch.int32, torch.int64, torch.uint8, torch.float32
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is None:
        return _raw_stream(torch._C._cuda_getDevice()) if _raw_stream else torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t: torch.Tensor, dtype, name: str) -> int:
    if t.dtype is dtype and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    raise ValueError(f"{name}: expected a contiguous tensor")


def _heads(t: torch.Tensor, name: str):
    """Pointer and (token, head) strides of a bf16 [T, heads, dim] view with contiguous dims."""
    st = t.stride()
    if t.dtype is _bf16 and t.is_cuda and len(st) == 3 and st[2] == 1:
        return t.data_ptr(), st[0], st[1]
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    if t.dtype is not _bf16:
        raise ValueError(f"{name}: expected {_bf16}, got {t.dtype}")
    raise ValueError(f"{name}: expected [tokens, heads, dim] with contiguous dims")


def _want(t: torch.Tensor, shape: tuple, name: str) -> None:
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


class KVCache:
    """The paged E4M3 cache (codes and scale bytes as uint8 tensors):
    k [num_blocks, kv_heads, block_size/16, head_dim/16, 16 tokens, 16 dims],
    v [num_blocks, kv_heads, block_size/16, head_dim, 16 tokens],
    k_scale, v_scale [num_blocks, kv_heads]."""
    __slots__ = ("k", "v", "k_scale", "v_scale", "num_blocks", "kv_heads", "head_dim", "block_size", "_c", "_ref")

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor):
        if k.dim() != 6:
            raise ValueError(f"k: expected six axes, got {tuple(k.shape)}")
        nb, heads, subs, chunks = k.shape[:4]
        _want(k, (nb, heads, subs, chunks, 16, 16), "k")
        _want(v, (nb, heads, subs, 16 * chunks, 16), "v")
        _want(k_scale, (nb, heads), "k_scale")
        _want(v_scale, (nb, heads), "v_scale")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_blocks, self.kv_heads, self.head_dim, self.block_size = nb, heads, 16 * chunks, 16 * subs
        self._c = _Cache(_ptr(k, _u8, "k"), _ptr(v, _u8, "v"), _ptr(k_scale, _u8, "k_scale"), _ptr(v_scale, _u8, "v_scale"), nb, heads,
                         16 * chunks, 16 * subs)
        self._ref = C.byref(self._c)

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
    __slots__ = ("codes", "scale", "n", "k", "_codes", "_scale")

    def __init__(self, codes: torch.Tensor, scale: torch.Tensor):
        self.n, self.k = codes.shape
        _want(scale, (-(-self.n // 128), -(-self.k // 128)), "scale")
        self.codes, self.scale = codes, scale
        self._codes, self._scale = _ptr(codes, _u8, "codes"), _ptr(scale, _u8, "scale")

    @staticmethod
    def from_dense(w: torch.Tensor, stream=None) -> "FP8Weight":
        """Quantises w bf16 [N, K] (moe_quantize_fp8_weight)."""
        n, k = w.shape
        out = FP8Weight(torch.empty((n, k), dtype=torch.uint8, device=w.device),
                        torch.empty((-(-n // 128), -(-k // 128)), dtype=torch.uint8, device=w.device))
        moe_quantize_fp8_weight(w, out, stream)
        return out


def alloc_workspace(max_tokens: int, max_requests: int, q_heads: int, cache: KVCache, weights=()) -> torch.Tensor:
    """A workspace for steps of up to these sizes: the attention's and, for
    ``weights`` (FP8Weight), the projections'."""
    n = max([512, moe_kv_attention_workspace_size(max_tokens, max_requests, q_heads, cache.kv_heads, cache.head_dim)] +
            [moe_linear_fp8_workspace_size(max_tokens, *w.codes.shape) for w in weights])
    ws = torch.empty(n, dtype=torch.uint8, device=cache.k.device)
    with torch.cuda.device(ws.device):
        moe.moe_workspace_init(ws)
    return ws


def moe_kv_build_tables(ctx_lens, new_lens, block_size, free_blocks, free_head, block_table, kv_lens, q_offsets, slot_map,
                        positions, free_head_out, ws, stream=None):
    B, T = ctx_lens.numel(), slot_map.numel()
    if new_lens.numel() != B or kv_lens.numel() != B or q_offsets.numel() != B + 1 or positions.numel() != T or block_table.shape[0] != B:
        raise ValueError(f"expected {B} new_lens, kv_lens and rows of block_table, {B + 1} q_offsets, {T} positions")
    _check(lib().moe_kv_build_tables(_ptr(ctx_lens, _i32, "ctx_lens"), _ptr(new_lens, _i32, "new_lens"), B, T, block_size,
                                     _ptr(free_blocks, _i32, "free_blocks"), free_blocks.numel(),
                                     _ptr(free_head, _i32, "free_head"), _ptr(block_table, _i32, "block_table"),
                                     block_table.shape[1], _ptr(kv_lens, _i32, "kv_lens"), _ptr(q_offsets, _i32, "q_offsets"),
                                     _ptr(slot_map, _i64, "slot_map"), _ptr(positions, _i32, "positions"),
                                     _ptr(free_head_out, _i32, "free_head_out"), _ptr(ws, _u8, "ws"), ws.numel(),
                                     _stream(stream)), "moe_kv_build_tables")


def moe_kv_append(k, v, slot_map, cache: KVCache, ws, stream=None):
    """k, v bf16 [T, kv_heads, head_dim]; views with strides are taken as they are."""
    T = slot_map.numel()
    _want(k, (T, cache.kv_heads, cache.head_dim), "k")
    _want(v, (T, cache.kv_heads, cache.head_dim), "v")
    _check(lib().moe_kv_append(*_heads(k, "k"), *_heads(v, "v"), _ptr(slot_map, _i64, "slot_map"), T, cache._ref,
                               _ptr(ws, _u8, "ws"), ws.numel(), _stream(stream)), "moe_kv_append")


def moe_kv_attention_workspace_size(T: int, B: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    return int(lib().moe_kv_attention_workspace_size(T, B, q_heads, kv_heads, head_dim))


def moe_kv_attention(q, cache: KVCache, block_table, q_offsets, kv_lens, softmax_scale, out, lse, ws, causal=True, window=0,
                     stream=None):
    """q bf16 [T, q_heads, head_dim] (strided views are taken as they are), out
    bf16 of the same shape, contiguous; lse fp32 [T, q_heads] or None."""
    shape, B = q.shape, kv_lens.numel()
    if len(shape) != 3 or shape[2] != cache.head_dim:
        raise ValueError(f"q: expected [tokens, heads, {cache.head_dim}], got {tuple(shape)}")
    T, q_heads = shape[0], shape[1]
    _want(out, shape, "out")
    if lse is not None:
        _want(lse, (T, q_heads), "lse")
    if q_offsets.numel() != B + 1 or block_table.shape[0] != B:
        raise ValueError(f"expected {B + 1} q_offsets and {B} rows of block_table")
    _check(lib().moe_kv_attention(*_heads(q, "q"), T, q_heads, cache._ref, _ptr(block_table, _i32, "block_table"),
                                  block_table.shape[1], _ptr(q_offsets, _i32, "q_offsets"), _ptr(kv_lens, _i32, "kv_lens"), B,
                                  softmax_scale, causal, window, _ptr(out, _bf16, "out"),
                                  None if lse is None else _ptr(lse, _f32, "lse"), _ptr(ws, _u8, "ws"), ws.numel(),
                                  _stream(stream)), "moe_kv_attention")


def moe_quantize_fp8_weight(w, out: FP8Weight, stream=None):
    _want(w, (out.n, out.k), "w")
    _check(lib().moe_quantize_fp8_weight(_ptr(w, _bf16, "w"), out.n, out.k, out._codes, out._scale, _stream(stream)),
           "moe_quantize_fp8_weight")


def moe_linear_fp8_workspace_size(T: int, N: int, K: int) -> int:
    return int(lib().moe_linear_fp8_workspace_size(T, N, K))


def moe_linear_fp8(x, w: FP8Weight, y, ws, stream=None):
    """y bf16 [T, N] = x W^T; x bf16 [T, K], rows may lie further apart than K."""
    st, T = x.stride(), x.shape[0]
    if not x.is_cuda or x.dtype is not _bf16 or len(st) != 2 or st[1] != 1:
        raise ValueError("x: expected a CUDA bf16 matrix with contiguous rows")
    _want(x, (T, w.k), "x")
    _want(y, (T, w.n), "y")
    _check(lib().moe_linear_fp8(x.data_ptr(), st[0] if T > 1 else w.k, T, w._codes, w._scale, w.n, w.k, _ptr(y, _bf16, "y"),
                                _ptr(ws, _u8, "ws"), ws.numel(), _stream(stream)), "moe_linear_fp8")
