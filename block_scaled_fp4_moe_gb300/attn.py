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
import dataclasses

import torch

from . import moe
from .moe import _check, _ptr, _stream


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


def _heads(t: torch.Tensor, dtype, name: str):
    """Pointer and (token, head) strides of a [T, heads, dim] view with contiguous dims."""
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.dim() != 3 or t.stride(2) != 1:
        raise ValueError(f"{name}: expected [tokens, heads, dim] with contiguous dims")
    return C.c_void_p(t.data_ptr()), t.stride(0), t.stride(1)


def _want(t: torch.Tensor, shape, name: str) -> None:
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


@dataclasses.dataclass
class KVCache:
    """The paged E4M3 cache (codes and scale bytes as uint8 tensors):
    k [num_blocks, kv_heads, block_size/16, head_dim/16, 16 tokens, 16 dims],
    v [num_blocks, kv_heads, block_size/16, head_dim, 16 tokens],
    k_scale, v_scale [num_blocks, kv_heads]."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor

    def __post_init__(self):
        nb, heads, subs, chunks = self.k.shape[:4]
        _want(self.k, (nb, heads, subs, chunks, 16, 16), "k")
        _want(self.v, (nb, heads, subs, 16 * chunks, 16), "v")
        _want(self.k_scale, (nb, heads), "k_scale")
        _want(self.v_scale, (nb, heads), "v_scale")
        u8 = torch.uint8
        self._c = _Cache(_ptr(self.k, u8, "k").value, _ptr(self.v, u8, "v").value, _ptr(self.k_scale, u8, "k_scale").value,
                         _ptr(self.v_scale, u8, "v_scale").value, nb, heads, 16 * chunks, 16 * subs)

    @staticmethod
    def empty(num_blocks: int, kv_heads: int, head_dim: int, block_size: int, device="cuda") -> "KVCache":
        """A cache whose blocks hold nothing yet (its memory is not cleared)."""
        def make(*shape):
            return torch.empty(shape, dtype=torch.uint8, device=device)
        subs = block_size // 16
        return KVCache(make(num_blocks, kv_heads, subs, head_dim // 16, 16, 16), make(num_blocks, kv_heads, subs, head_dim, 16),
                       make(num_blocks, kv_heads), make(num_blocks, kv_heads))

    @property
    def kv_heads(self) -> int:
        return self.k.shape[1]

    @property
    def head_dim(self) -> int:
        return self.v.shape[3]

    @property
    def block_size(self) -> int:
        return 16 * self.v.shape[2]


@dataclasses.dataclass
class FP8Weight:
    """codes uint8 [N, K] (E4M3) and scale uint8 [ceil(N/128), ceil(K/128)] (E8M0)."""
    codes: torch.Tensor
    scale: torch.Tensor

    def __post_init__(self):
        n, k = self.codes.shape
        _want(self.scale, (-(-n // 128), -(-k // 128)), "scale")

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
    i32 = torch.int32
    B, T = ctx_lens.numel(), slot_map.numel()
    _want(new_lens, (B,), "new_lens")
    _want(kv_lens, (B,), "kv_lens")
    _want(q_offsets, (B + 1,), "q_offsets")
    _want(positions, (T,), "positions")
    if block_table.shape[0] != B:
        raise ValueError(f"block_table: expected {B} rows, got {block_table.shape[0]}")
    _check(lib().moe_kv_build_tables(_ptr(ctx_lens, i32, "ctx_lens"), _ptr(new_lens, i32, "new_lens"), B, T, block_size,
                                     _ptr(free_blocks, i32, "free_blocks"), free_blocks.numel(),
                                     _ptr(free_head, i32, "free_head"), _ptr(block_table, i32, "block_table"),
                                     block_table.shape[1], _ptr(kv_lens, i32, "kv_lens"), _ptr(q_offsets, i32, "q_offsets"),
                                     _ptr(slot_map, torch.int64, "slot_map"), _ptr(positions, i32, "positions"),
                                     _ptr(free_head_out, i32, "free_head_out"), _ptr(ws, torch.uint8, "ws"), ws.numel(),
                                     _stream(stream)), "moe_kv_build_tables")


def moe_kv_append(k, v, slot_map, cache: KVCache, ws, stream=None):
    """k, v bf16 [T, kv_heads, head_dim]; views with strides are taken as they are."""
    T = k.shape[0]
    _want(k, (T, cache.kv_heads, cache.head_dim), "k")
    _want(v, k.shape, "v")
    _want(slot_map, (T,), "slot_map")
    _check(lib().moe_kv_append(*_heads(k, torch.bfloat16, "k"), *_heads(v, torch.bfloat16, "v"),
                               _ptr(slot_map, torch.int64, "slot_map"), T, C.byref(cache._c), _ptr(ws, torch.uint8, "ws"),
                               ws.numel(), _stream(stream)), "moe_kv_append")


def moe_kv_attention_workspace_size(T: int, B: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    return int(lib().moe_kv_attention_workspace_size(T, B, q_heads, kv_heads, head_dim))


def moe_kv_attention(q, cache: KVCache, block_table, q_offsets, kv_lens, softmax_scale, out, lse, ws, causal=True, window=0,
                     stream=None):
    """q bf16 [T, q_heads, head_dim] (strided views are taken as they are), out
    bf16 of the same shape, contiguous; lse fp32 [T, q_heads] or None."""
    T, q_heads = q.shape[:2]
    B = kv_lens.numel()
    _want(q, (T, q_heads, cache.head_dim), "q")
    _want(out, q.shape, "out")
    _want(q_offsets, (B + 1,), "q_offsets")
    if lse is not None:
        _want(lse, (T, q_heads), "lse")
    if block_table.shape[0] != B:
        raise ValueError(f"block_table: expected {B} rows, got {block_table.shape[0]}")
    i32 = torch.int32
    _check(lib().moe_kv_attention(*_heads(q, torch.bfloat16, "q"), T, q_heads, C.byref(cache._c),
                                  _ptr(block_table, i32, "block_table"), block_table.shape[1],
                                  _ptr(q_offsets, i32, "q_offsets"), _ptr(kv_lens, i32, "kv_lens"), B, float(softmax_scale),
                                  int(causal), int(window), _ptr(out, torch.bfloat16, "out"),
                                  _ptr(lse, torch.float32, "lse"), _ptr(ws, torch.uint8, "ws"), ws.numel(),
                                  _stream(stream)), "moe_kv_attention")


def moe_quantize_fp8_weight(w, out: FP8Weight, stream=None):
    n, k = w.shape
    _want(out.codes, (n, k), "codes")
    _check(lib().moe_quantize_fp8_weight(_ptr(w, torch.bfloat16, "w"), n, k, _ptr(out.codes, torch.uint8, "codes"),
                                         _ptr(out.scale, torch.uint8, "scale"), _stream(stream)), "moe_quantize_fp8_weight")


def moe_linear_fp8_workspace_size(T: int, N: int, K: int) -> int:
    return int(lib().moe_linear_fp8_workspace_size(T, N, K))


def moe_linear_fp8(x, w: FP8Weight, y, ws, stream=None):
    """y bf16 [T, N] = x W^T; x bf16 [T, K], rows may lie further apart than K."""
    T, K = x.shape
    N = w.codes.shape[0]
    if not x.is_cuda or x.dtype != torch.bfloat16 or x.stride(1) != 1:
        raise ValueError("x: expected a CUDA bf16 tensor with contiguous rows")
    _want(w.codes, (N, K), "codes")
    _want(y, (T, N), "y")
    _check(lib().moe_linear_fp8(C.c_void_p(x.data_ptr()), x.stride(0) if T > 1 else K, T, _ptr(w.codes, torch.uint8, "codes"),
                                _ptr(w.scale, torch.uint8, "scale"), N, K, _ptr(y, torch.bfloat16, "y"),
                                _ptr(ws, torch.uint8, "ws"), ws.numel(), _stream(stream)), "moe_linear_fp8")
