"""The operators a decoding step runs around the quantized layers (C ABI in
``include/flexq_serve.h``), bound the same way as the layers themselves: arguments are
checked, outputs and workspaces allocated when the caller brings none, and the
work runs in the HIP kernels on the current stream of the tensors' GPU.  For the calls
that run once a layer and step the checks are in ``_serve.so`` (csrc/serve_binding.cpp).

* :func:`pack_w4`, :func:`gemv_w4`, :class:`W4Linear`  4-bit group-scaled weights and
  their product with a few activation rows (fp16 or bf16)
* :func:`block_tables`     a paged cache's block tables and slot maps from lengths
* :func:`kv_cache`, :func:`kv_cache_write`  the paged cache and the writing of new tokens
* :func:`tree_attention`   attention of drafted tokens (one token, a chain or a tree)
  over the paged cache
* :func:`kv4_cache`, :func:`kv4_cache_write`, :func:`kv4_cache_read`, :func:`kv4_attention`
  the same over a cache of 4-bit codes, with an optional sliding window
* :func:`lora_add`         low-rank adapters of many requests, added to a layer's output
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

import torch

import w6a6_w6a8_integer_amd as _fq

_P, _I64, _I32, _SZ, _F = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t,
                           ctypes.c_float)
# (restype, argtypes) of every symbol include/flexq_serve.h declares
SIGNATURES = {
    "flexq_packed_w4_bytes": (_SZ, [_I64, _I64]),
    "flexq_pack_w4": (ctypes.c_int, [_P, _I32, _I64, _I64, _I32, _P, _P, _P]),
    "flexq_gemv_w4": (ctypes.c_int, [_P, _I32, _I64, _P, _P, _I64, _I64, _I64, _I32, _P, _SZ, _P,
                                     _P]),
    "flexq_gemv_w4_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "flexq_block_tables": (ctypes.c_int, [_P, _P, _I64, _P, _I64, _P, _I32, _P, _I64, _I64, _P,
                                          _P, _P, _P]),
    "flexq_kv_cache_write": (ctypes.c_int, [_P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I64, _I64,
                                            _I64, _I32, _P, _P, _P]),
    "flexq_tree_attention": (ctypes.c_int, [_P, _I32, _I64, _I64, _P, _P, _I64, _I32, _P, _I64,
                                            _P, _P, _I64, _I64, _I64, _I64, _I64, _I64, _P, _I64,
                                            _F, _P, _SZ, _P, _P, _P]),
    "flexq_tree_attention_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I64, _I64]),
    "flexq_kv4_cache_write": (ctypes.c_int, [_P, _I64, _I64, _P, _I64, _I64, _I32, _P, _I64, _I64,
                                             _I64, _I64, _I32, _P, _P, _P, _P]),
    "flexq_kv4_cache_read": (ctypes.c_int, [_P, _P, _P, _P, _I64, _I64, _I64, _I64, _I32, _I32, _P,
                                            _P, _P]),
    "flexq_kv4_attention": (ctypes.c_int, [_P, _I32, _I64, _I64, _P, _P, _P, _I64, _I32, _P, _I64,
                                           _P, _P, _I64, _I64, _I64, _I64, _I64, _I64, _P, _I64,
                                           _I64, _I64, _F, _P, _SZ, _P, _P, _P]),
    "flexq_kv4_attention_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I64, _I64]),
    "flexq_lora_add": (ctypes.c_int, [_P, _I32, _I64, _P, _I64, _P, _P, _P, _P, _P, _I64, _I64,
                                      _I64, _I64, _I64, _P, _SZ, _P, _I64, _P]),
    "flexq_lora_add_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I64, _I64]),
}

_DTYPE = {torch.float16: 0, torch.bfloat16: 1}
PAGE_SIZES = (16, 32, 64, 128, 256)
HEAD_WIDTHS = (64, 96, 128, 256)


def _dtype(t, name: str) -> int:
    code = _DTYPE.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if code is None:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
        raise TypeError(f"{name} must be float16 or bfloat16, got {t.dtype}")
    return code


_calls = None


def _native():
    """The functions of _serve.so, bound to the loaded library."""
    global _calls
    if _calls is None:
        lib = _fq.lib()
        path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_serve.so")
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is not built: run __graft_entry__.build() "
                               "(there is no fallback)")
        spec = importlib.util.spec_from_file_location(f"{__package__}._serve", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.bind(*(ctypes.cast(getattr(lib, f"flexq_{name}"), ctypes.c_void_p).value
                      for name in ("gemv_w4", "gemv_w4_workspace_bytes", "block_tables",
                                   "kv_cache_write", "tree_attention",
                                   "tree_attention_workspace_bytes", "kv4_cache_write",
                                   "kv4_cache_read", "kv4_attention",
                                   "kv4_attention_workspace_bytes", "lora_add",
                                   "lora_add_workspace_bytes")))
        _calls = module
    return _calls


def _call(name: str, dev, *args):
    """The C call on the current stream of `dev`, with that GPU current."""
    fn = getattr(_fq.lib(), name)
    stream = torch.cuda.current_stream(dev).cuda_stream
    if torch.cuda.current_device() == dev.index:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, stream)
    if status != 0:
        raise _fq.FlexqError(status, name)


def _group(group: int) -> int:
    if group not in (32, 64, 128):
        raise ValueError(f"group = {group} must be 32, 64 or 128")
    return group


def _packed4(w4, N: int, K: int):
    if isinstance(w4, torch.Tensor) and w4.dim() != 1:
        raise ValueError(f"w4 must be 1-D, got shape {tuple(w4.shape)}")
    return _fq._tensor(w4, torch.int32, "w4", min_bytes=N * K // 2)


def pack_w4(w: torch.Tensor, group: int = 128, w4: torch.Tensor | None = None,
            s_w: torch.Tensor | None = None):
    """W[N][K] (fp16 or bf16) -> (w4 int32[N*K/8] holding the packed codes, s_w
    fp16[K/group][N], group-major)."""
    code = _dtype(w, "w")
    _fq._matrix(w, w.dtype, "w")
    N, K = w.shape
    _fq._groups(K, "pack_w4")
    _fq._cols(N)
    G = K // _group(group)
    if w4 is None:
        w4 = torch.empty(max(1, N * K // 8), dtype=torch.int32, device=w.device)
    if s_w is None:
        s_w = torch.empty((G, N), dtype=torch.float16, device=w.device)
    _packed4(w4, N, K)
    _fq._tensor(s_w, torch.float16, "s_w", shape=(G, N))
    dev = _fq._on_gpu(w=w, w4=w4, s_w=s_w)
    _call("flexq_pack_w4", dev, w.data_ptr(), code, N, K, group, w4.data_ptr(), s_w.data_ptr())
    return w4, s_w


def gemv_w4_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(_fq.lib().flexq_gemv_w4_workspace_bytes(M, N, K))


def gemv_w4(x: torch.Tensor, w4: torch.Tensor, s_w: torch.Tensor, N: int,
            y: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """Y[M][N] = X[M][K] times the 4-bit weights (flexq_gemv_w4), X and Y fp16 or bf16,
    X's rows contiguous (they may be strided); the group size is K / len(s_w).  Meant for
    few rows: the weights are read once per 64 of them."""
    return (_calls or _native()).gemv_w4(x, w4, s_w, N, y, workspace)


class W4Linear:
    """A weight-only 4-bit nn.Linear-shaped layer for a few activation rows."""

    def __init__(self, weight: torch.Tensor, group: int = 128):
        self.N, self.K = weight.shape
        self.w4, self.s_w = pack_w4(weight.contiguous(), group)

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        return gemv_w4(x, self.w4, self.s_w, self.N)


def block_tables(ctx_lens: torch.Tensor, new_lens: torch.Tensor, free_pages: torch.Tensor,
                 block_table: torch.Tensor, page_size: int, max_tokens: int,
                 free_head: torch.Tensor | None = None, slot_map: torch.Tensor | None = None,
                 cu_new: torch.Tensor | None = None, counts: torch.Tensor | None = None):
    """A step's block tables and slot map (flexq_block_tables), all int32: request b
    holds ctx_lens[b] tokens and gets new_lens[b] more; pages it lacks are taken from
    free_pages in order of the requests, from *free_head on (0 where it is None), and
    entered into block_table[B][max_blocks] in place.  Returns (slot_map[max_tokens],
    cu_new[B + 1], counts[3]); counts = new tokens, pages taken, next free head.  Slots
    past the new tokens, and of tokens no page was left for, are -1."""
    return (_calls or _native()).block_tables(ctx_lens, new_lens, free_pages, block_table,
                                              page_size, max_tokens, free_head, slot_map, cu_new,
                                              counts)


def kv_cache(num_pages: int, Hkv: int, D: int, page_size: int, dtype=torch.float16,
             device="cuda"):
    """An empty paged cache: (keys [pages][Hkv][page_size/16][D/32][16][32], values
    [pages][Hkv][page_size/16][D][16])."""
    if page_size not in PAGE_SIZES or D not in HEAD_WIDTHS:
        raise ValueError(f"page_size must be one of {PAGE_SIZES} and D one of {HEAD_WIDTHS}")
    k = torch.empty((num_pages, Hkv, page_size // 16, D // 32, 16, 32), dtype=dtype, device=device)
    v = torch.empty((num_pages, Hkv, page_size // 16, D, 16), dtype=dtype, device=device)
    return k, v


def kv_cache_write(k: torch.Tensor, v: torch.Tensor, slot_map: torch.Tensor,
                   k_cache: torch.Tensor, v_cache: torch.Tensor):
    """Keys and values k, v [T][Hkv][D] into the paged cache at the slots
    slot_map int32[T] (flexq_kv_cache_write); negative slots drop their token.  k and v may
    be strided over tokens and heads, as slices of a fused projection's output are."""
    (_calls or _native()).kv_cache_write(k, v, slot_map, k_cache, v_cache)


def tree_attention_workspace_bytes(B: int, max_new: int, H: int, Hkv: int, D: int) -> int:
    return int(_fq.lib().flexq_tree_attention_workspace_bytes(B, max_new, H, Hkv, D))


def tree_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   block_table: torch.Tensor, ctx_lens: torch.Tensor, cu_new: torch.Tensor,
                   tree_mask: torch.Tensor | None = None, scale: float | None = None,
                   max_new: int | None = None, out: torch.Tensor | None = None,
                   lse: torch.Tensor | None = None, return_lse: bool = False,
                   workspace: torch.Tensor | None = None):
    """Attention of drafted tokens over the paged cache (flexq_tree_attention).

    q [T][H][D] (may be strided over tokens and heads) holds the new tokens of all
    requests, request b's at rows cu_new[b] .. cu_new[b + 1] - 1; their keys and values
    are already in the cache behind the request's ctx_lens[b] others.  tree_mask int32
    [T][words]: bit j of a token's words lets it attend the request's drafted token j;
    None is a chain (j up to the token itself).  max_new bounds the new tokens of one
    request (further ones are not computed); left out it is T, or the bits of a mask if
    those are fewer.  The call is laid out for that many, so pass what a step really has:
    32 single tokens of 64 heads on 8 over 4k take 105 us without it and 54 with it.  Returns out [T][H][D], or (out, lse fp32[T][H]) where lse is
    asked for."""
    return (_calls or _native()).tree_attention(q, k_cache, v_cache, block_table, ctx_lens,
                                                cu_new, tree_mask, scale, max_new, out, lse,
                                                return_lse, workspace)


def kv4_cache(num_pages: int, Hkv: int, D: int, page_size: int, device="cuda"):
    """An empty paged cache of 4-bit codes, for fp16 and bf16 models alike: (k_codes int32
    [pages][Hkv][page_size/16][16][D/8], v_codes int32 [pages][Hkv][page_size/16][2][D/2][2],
    scales fp16 [pages][Hkv][page_size/16][4][16])."""
    if page_size not in PAGE_SIZES or D not in HEAD_WIDTHS:
        raise ValueError(f"page_size must be one of {PAGE_SIZES} and D one of {HEAD_WIDTHS}")
    lead = (num_pages, Hkv, page_size // 16)
    return (torch.empty((*lead, 16, D // 8), dtype=torch.int32, device=device),
            torch.empty((*lead, 2, D // 2, 2), dtype=torch.int32, device=device),
            torch.empty((*lead, 4, 16), dtype=torch.float16, device=device))


def kv4_cache_write(k: torch.Tensor, v: torch.Tensor, slot_map: torch.Tensor,
                    k_codes: torch.Tensor, v_codes: torch.Tensor, scales: torch.Tensor):
    """Keys and values k, v [T][Hkv][D] into the 4-bit cache at the slots slot_map int32[T]
    (flexq_kv4_cache_write), each token and head with a scale and an offset of its own; negative
    slots drop their token, and the others should differ.  k and v may be strided over tokens
    and heads."""
    (_calls or _native()).kv4_cache_write(k, v, slot_map, k_codes, v_codes, scales)


def kv4_cache_read(slot_map: torch.Tensor, k_codes: torch.Tensor, v_codes: torch.Tensor,
                   scales: torch.Tensor, dtype=torch.float16, k: torch.Tensor | None = None,
                   v: torch.Tensor | None = None):
    """The cache's tokens at slot_map int32[T] as rows of `dtype` (flexq_kv4_cache_read): what
    :func:`kv4_attention` sees of them.  Slots outside the cache read as 0.  Returns (k, v)
    [T][Hkv][D]."""
    return (_calls or _native()).kv4_cache_read(slot_map, k_codes, v_codes, scales, dtype, k, v)


def kv4_attention_workspace_bytes(B: int, max_new: int, H: int, Hkv: int, D: int) -> int:
    return int(_fq.lib().flexq_kv4_attention_workspace_bytes(B, max_new, H, Hkv, D))


def kv4_attention(q: torch.Tensor, k_codes: torch.Tensor, v_codes: torch.Tensor,
                  scales: torch.Tensor, block_table: torch.Tensor, ctx_lens: torch.Tensor,
                  cu_new: torch.Tensor, tree_mask: torch.Tensor | None = None,
                  scale: float | None = None, max_new: int | None = None,
                  window: int | None = None, sinks: int = 0, out: torch.Tensor | None = None,
                  lse: torch.Tensor | None = None, return_lse: bool = False,
                  workspace: torch.Tensor | None = None):
    """:func:`tree_attention` over the 4-bit cache (flexq_kv4_attention), q fp16 or bf16.

    With a window a token attends the last `window` positions, its own among them, and the
    first `sinks` of its request; keys between, before every window of the request's tokens, are
    not read (a prompt that begins within its window reads its keys from the first on for
    every block of rows).  In a tree the drafted tokens that a token attends are the last of its
    window's positions, and are attended whatever the window."""
    return (_calls or _native()).kv4_attention(q, k_codes, v_codes, scales, block_table, ctx_lens,
                                               cu_new, tree_mask, scale, max_new, window, sinks,
                                               out, lse, return_lse, workspace)


def lora_add_workspace_bytes(T: int, N: int, K: int, R: int, L: int) -> int:
    return int(_fq.lib().flexq_lora_add_workspace_bytes(T, N, K, R, L))


def lora_add(x: torch.Tensor, y: torch.Tensor, adapters: torch.Tensor, a: torch.Tensor,
             b: torch.Tensor, ranks: torch.Tensor | None = None,
             scales: torch.Tensor | None = None, out: torch.Tensor | None = None,
             workspace: torch.Tensor | None = None):
    """The requests' own low-rank adapters beside a layer they share (flexq_lora_add): token t
    of x [T][K] with adapter i = adapters[t] (int32; none where that is outside [0, L)) adds
    scales[i] * b[i] (a[i] x[t]) to y[t] [N], a [L][R][K] and b [L][N][R] of which the first
    ranks[i] rows and columns count (all R where ranks is None).  x and y are fp16 or bf16 and may
    be strided rows.  In place on y unless `out` is given; returns it.  There is no backward
    pass: with gradients enabled, tensors that require them are refused."""
    return (_calls or _native()).lora_add(x, y, adapters, a, b, ranks, scales, out, workspace)
