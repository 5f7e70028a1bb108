"""The operators a decoding step runs around the quantized layers (C ABI in
``include/flexq_serve.h``), bound the same way as the layers themselves: arguments are
checked here, outputs and workspaces allocated when the caller brings none, and the
work runs in the HIP kernels on the current stream of the tensors' GPU.

* :func:`pack_w4`, :func:`gemv_w4`, :class:`W4Linear`  4-bit group-scaled weights and
  their product with a few activation rows (fp16 or bf16)
* :func:`block_tables`     a paged cache's block tables and slot maps from lengths
* :func:`kv_cache`, :func:`kv_cache_write`  the paged cache and the writing of new tokens
* :func:`tree_attention`   attention of drafted tokens (one token, a chain or a tree)
  over the paged cache
"""
from __future__ import annotations

import ctypes
import math

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


def _rows(t, dtype, name: str, dims: int):
    """A tensor whose last dimension is contiguous; the others may be strided."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != dims:
        raise ValueError(f"{name} must be {dims}-D, got shape {tuple(t.shape)}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")
    return t


def _int32(t, name: str, shape):
    return _fq._tensor(t, torch.int32, name, shape=shape)


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


def _workspace(t, need: int):
    if isinstance(t, torch.Tensor) and t.dim() != 1:
        raise ValueError(f"workspace must be 1-D, got shape {tuple(t.shape)}")
    return _fq._tensor(t, torch.uint8, "workspace", min_bytes=need)


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
    code = _dtype(x, "x")
    _rows(x, x.dtype, "x", 2)
    M, K = x.shape
    _fq._groups(K, "gemv_w4")
    N = _fq._cols(N)
    if not isinstance(s_w, torch.Tensor) or s_w.dim() != 2:
        raise ValueError("s_w must be a 2-D tensor [K/group][N]")
    G = s_w.shape[0]
    if G <= 0 or K % G:
        raise ValueError(f"s_w must have K / group rows for K = {K}, got {G}")
    _group(K // G)
    _fq._tensor(s_w, torch.float16, "s_w", shape=(G, N))
    _packed4(w4, N, K)
    if y is None:
        y = torch.empty((M, N), dtype=x.dtype, device=x.device)
    _fq._tensor(y, x.dtype, "y", shape=(M, N))
    need = gemv_w4_workspace_bytes(M, N, K)
    tensors = dict(x=x, w4=w4, s_w=s_w, y=y)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    if workspace is not None:
        tensors["workspace"] = _workspace(workspace, need)
    dev = _fq._on_gpu(**tensors)
    _call("flexq_gemv_w4", dev, x.data_ptr(), code, x.stride(0), w4.data_ptr(), s_w.data_ptr(), M,
          N, K, K // G, workspace.data_ptr() if workspace is not None else None,
          workspace.numel() if workspace is not None else 0, y.data_ptr())
    return y


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
    if isinstance(block_table, torch.Tensor) and block_table.dim() != 2:
        raise ValueError(f"block_table must be 2-D, got shape {tuple(block_table.shape)}")
    _fq._tensor(block_table, torch.int32, "block_table")
    B, max_blocks = block_table.shape
    dev = block_table.device
    _int32(ctx_lens, "ctx_lens", (B,))
    _int32(new_lens, "new_lens", (B,))
    if isinstance(free_pages, torch.Tensor) and free_pages.dim() != 1:
        raise ValueError(f"free_pages must be 1-D, got shape {tuple(free_pages.shape)}")
    _fq._tensor(free_pages, torch.int32, "free_pages")
    max_tokens = int(max_tokens)
    if max_tokens < 0:
        raise ValueError(f"max_tokens = {max_tokens} must not be negative")
    if slot_map is None:
        slot_map = torch.empty(max_tokens, dtype=torch.int32, device=dev)
    if cu_new is None:
        cu_new = torch.empty(B + 1, dtype=torch.int32, device=dev)
    if counts is None:
        counts = torch.empty(3, dtype=torch.int32, device=dev)
    _int32(slot_map, "slot_map", (max_tokens,))
    _int32(cu_new, "cu_new", (B + 1,))
    _int32(counts, "counts", (3,))
    tensors = dict(block_table=block_table, ctx_lens=ctx_lens, new_lens=new_lens,
                   free_pages=free_pages, slot_map=slot_map, cu_new=cu_new, counts=counts)
    if free_head is not None:
        tensors["free_head"] = _int32(free_head, "free_head", (1,))
    dev = _fq._on_gpu(**tensors)
    _call("flexq_block_tables", dev, ctx_lens.data_ptr(), new_lens.data_ptr(), B,
          free_pages.data_ptr(), free_pages.numel(),
          free_head.data_ptr() if free_head is not None else None, page_size,
          block_table.data_ptr(), max_blocks, max_tokens, slot_map.data_ptr(), cu_new.data_ptr(),
          counts.data_ptr())
    return slot_map, cu_new, counts


def kv_cache(num_pages: int, Hkv: int, D: int, page_size: int, dtype=torch.float16,
             device="cuda"):
    """An empty paged cache: (keys [pages][Hkv][page_size/16][D/32][16][32], values
    [pages][Hkv][page_size/16][D][16])."""
    if page_size not in PAGE_SIZES or D not in HEAD_WIDTHS:
        raise ValueError(f"page_size must be one of {PAGE_SIZES} and D one of {HEAD_WIDTHS}")
    k = torch.empty((num_pages, Hkv, page_size // 16, D // 32, 16, 32), dtype=dtype, device=device)
    v = torch.empty((num_pages, Hkv, page_size // 16, D, 16), dtype=dtype, device=device)
    return k, v


def _cache(k_cache, v_cache, dtype):
    """(pages, Hkv, D, page_size) of a paged cache."""
    if not isinstance(v_cache, torch.Tensor) or v_cache.dim() != 5:
        raise ValueError("v_cache must be a 5-D tensor [pages][Hkv][page_size/16][D][16]")
    pages, Hkv, blocks, D, last = v_cache.shape
    if last != 16 or D not in HEAD_WIDTHS or 16 * blocks not in PAGE_SIZES:
        raise ValueError(f"v_cache must be [pages][Hkv][page_size/16][D][16] with page_size one "
                         f"of {PAGE_SIZES} and D one of {HEAD_WIDTHS}, got "
                         f"{tuple(v_cache.shape)}")
    _fq._tensor(v_cache, dtype, "v_cache")
    _fq._tensor(k_cache, dtype, "k_cache", shape=(pages, Hkv, blocks, D // 32, 16, 32))
    return pages, Hkv, D, 16 * blocks


def kv_cache_write(k: torch.Tensor, v: torch.Tensor, slot_map: torch.Tensor,
                   k_cache: torch.Tensor, v_cache: torch.Tensor):
    """Keys and values k, v [T][Hkv][D] into the paged cache at the slots
    slot_map int32[T] (flexq_kv_cache_write); negative slots drop their token.  k and v may
    be strided over tokens and heads, as slices of a fused projection's output are."""
    _dtype(k, "k")
    _rows(k, k.dtype, "k", 3)
    pages, Hkv, D, page = _cache(k_cache, v_cache, k.dtype)
    T = k.shape[0]
    if tuple(k.shape) != (T, Hkv, D):
        raise ValueError(f"k must have shape {(T, Hkv, D)}, got {tuple(k.shape)}")
    _rows(v, k.dtype, "v", 3)
    if v.shape != k.shape:
        raise ValueError(f"v must have shape {tuple(k.shape)}, got {tuple(v.shape)}")
    _int32(slot_map, "slot_map", (T,))
    dev = _fq._on_gpu(k=k, v=v, slot_map=slot_map, k_cache=k_cache, v_cache=v_cache)
    _call("flexq_kv_cache_write", dev, k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(),
          v.stride(0), v.stride(1), slot_map.data_ptr(), T, Hkv, D, pages, page,
          k_cache.data_ptr(), v_cache.data_ptr())


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
    request (default: T).  Returns out [T][H][D], or (out, lse fp32[T][H]) where lse is
    asked for."""
    code = _dtype(q, "q")
    _rows(q, q.dtype, "q", 3)
    T, H, D = q.shape
    pages, Hkv, Dc, page = _cache(k_cache, v_cache, q.dtype)
    if Dc != D or Hkv <= 0 or H % Hkv:
        raise ValueError(f"q [{T}][{H}][{D}] does not fit a cache of {Hkv} heads of {Dc}")
    if isinstance(block_table, torch.Tensor) and block_table.dim() != 2:
        raise ValueError(f"block_table must be 2-D, got shape {tuple(block_table.shape)}")
    _fq._tensor(block_table, torch.int32, "block_table")
    B, max_blocks = block_table.shape
    _int32(ctx_lens, "ctx_lens", (B,))
    _int32(cu_new, "cu_new", (B + 1,))
    max_new = T if max_new is None else int(max_new)
    tensors = dict(q=q, k_cache=k_cache, v_cache=v_cache, block_table=block_table,
                   ctx_lens=ctx_lens, cu_new=cu_new)
    words = 0
    if tree_mask is not None:
        if isinstance(tree_mask, torch.Tensor) and tree_mask.dim() != 2:
            raise ValueError(f"tree_mask must be 2-D, got shape {tuple(tree_mask.shape)}")
        words = tree_mask.shape[1] if isinstance(tree_mask, torch.Tensor) else 0
        tensors["tree_mask"] = _int32(tree_mask, "tree_mask", (T, words))
        if max_new > 32 * words:
            raise ValueError(f"tree_mask has {32 * words} bits a token; max_new = {max_new}")
    dev = q.device
    if out is None:
        out = torch.empty((T, H, D), dtype=q.dtype, device=dev)
    tensors["out"] = _fq._tensor(out, q.dtype, "out", shape=(T, H, D))
    if lse is None and return_lse:
        lse = torch.empty((T, H), dtype=torch.float32, device=dev)
    if lse is not None:
        tensors["lse"] = _fq._tensor(lse, torch.float32, "lse", shape=(T, H))
    need = tree_attention_workspace_bytes(B, max_new, H, Hkv, D)
    if workspace is None:
        workspace = torch.empty(max(16, need), dtype=torch.uint8, device=dev)
    tensors["workspace"] = _workspace(workspace, need)
    dev = _fq._on_gpu(**tensors)
    _call("flexq_tree_attention", dev, q.data_ptr(), code, q.stride(0), q.stride(1),
          k_cache.data_ptr(), v_cache.data_ptr(), pages, page, block_table.data_ptr(), max_blocks,
          ctx_lens.data_ptr(), cu_new.data_ptr(), B, T, max_new, H, Hkv, D,
          tree_mask.data_ptr() if tree_mask is not None else None, words,
          1.0 / math.sqrt(D) if scale is None else float(scale), workspace.data_ptr(),
          workspace.numel(), out.data_ptr(), lse.data_ptr() if lse is not None else None)
    return out if lse is None else (out, lse)
