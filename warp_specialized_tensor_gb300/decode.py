"""Binding of the operators of a decoding step: the append to a paged cache with
the position rotation, attention of a step's tokens over the cache, products of few
rows with 4-bit weights (``include/wst.h`` has the definitions).

The functions are exported by the package.  They follow its conventions: the
C ABI's names, outputs passed in, sizes and strides read from the tensors, the
current stream unless one is given.
"""
from __future__ import annotations

import ctypes
import math

import torch

import warp_specialized_tensor_gb300 as _w
from warp_specialized_tensor_gb300.moe import _dense, _need, _rows, _stream, _type, _ws

__all__ = [
    "ROPE_HALVES", "ROPE_PAIRS", "wst_cache_append_bf16",
    "wst_tree_attention_bf16", "wst_tree_attention_workspace_size", "tree_attention_workspace",
    "wst_gemm_w4", "wst_grouped_gemm_w4", "wst_gemm_w4_workspace_size", "gemm_w4_workspace", "wst_gemm_w4_tile_rows",
]

# enum of include/wst.h
ROPE_HALVES, ROPE_PAIRS = 0, 1
_STYLES = {"halves": ROPE_HALVES, "pairs": ROPE_PAIRS}
_I32, _F32, _BF16 = torch.int32, torch.float32, torch.bfloat16


def declare(lib) -> None:
    """Argument types of the functions bound here."""
    P, I, L, Z, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_long, ctypes.c_size_t, ctypes.c_float
    for name, res, args in (
            ("wst_cache_append_bf16", I, [I, I, I, I, I, I, P, L, P, L, P, L, I, P, P, P, P, L, P, P, I, I, L, L, L, P, P]),
            ("wst_tree_attention_bf16", I, [I, I, I, I, I, P, L, P, P, P, I, L, P, P, I, I, L, L, L, P, I, L, F, P, L, I, P, Z, P]),
            ("wst_tree_attention_workspace_size", Z, []),
            ("wst_gemm_w4", I, [I, I, I, P, L, P, L, P, L, I, P, P, L, I, I, P, Z, P]),
            ("wst_grouped_gemm_w4", I, [I, I, I, I, P, L, P, L, L, P, L, L, I, P, P, L, P, L, I, I, P, Z, P]),
            ("wst_gemm_w4_workspace_size", Z, []),
            ("wst_gemm_w4_tile_rows", I, [I, I, I, I, I])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args


def _lib():
    return _w._lib or _w.load_library()


# As in the module's siblings, a good call pays for one look at each tensor; what is
# wrong is looked for only when that fails.
def _heads(t, name, dtype=None):
    """A CUDA tensor [T, heads, Dh] whose heads follow one another; returns the distance of its tokens."""
    if isinstance(t, torch.Tensor) and t.is_cuda and (dtype is None or t.dtype is dtype):
        shape, st = t.shape, t.stride()
        if len(st) == 3 and st[2] == 1 and st[1] == shape[2] and shape[0] > 1 and shape[1] > 0 and shape[2] > 1:
            return st[0]
    _need(t, name, dtype, (3,))
    T, H, Dh = t.shape
    if (H > 1 and t.stride(1) != Dh) or (Dh > 1 and t.stride(2) != 1):
        raise ValueError("%s must hold the heads of a token one after another" % name)
    per = 16 // t.element_size()
    return t.stride(0) if T > 1 else -(-max(H * Dh, 1) // per) * per


def _cache(k_cache, v_cache):
    """Checks the two arrays of a paged cache [pages, page_size, heads, Dh]; returns its shape and the strides of pages,
    tokens, heads."""
    if (isinstance(k_cache, torch.Tensor) and isinstance(v_cache, torch.Tensor) and k_cache.is_cuda and v_cache.is_cuda
            and k_cache.dtype is _BF16 and v_cache.dtype is _BF16):
        shape, st = k_cache.shape, k_cache.stride()
        if len(st) == 4 and st[3] == 1 and v_cache.stride() == st and v_cache.shape == shape and min(shape) > 1:
            return shape, st[0], st[1], st[2]
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, name, _BF16, (4,))
        if t.shape[3] > 1 and t.stride(3) != 1:
            raise ValueError("%s must have a contiguous last dimension" % name)
    if k_cache.shape != v_cache.shape or any(n > 1 and a != b for n, a, b in zip(k_cache.shape, k_cache.stride(), v_cache.stride())):
        raise ValueError("k_cache and v_cache must have the same shape and strides")
    (pages, page, heads, Dh), (sp, st, sh, _) = k_cache.shape, k_cache.stride()
    # (the stride of a dimension of one means nothing: one that every check takes)
    if heads == 1:
        sh = Dh
    if page == 1:
        st = heads * sh
    if pages == 1:
        sp = max(page * st, heads * sh)
    return k_cache.shape, sp, st, sh


# ----------------------------------------------------------------------------
# append
# ----------------------------------------------------------------------------
def wst_cache_append_bf16(k, v, positions, slots, k_cache, v_cache, inv_freq=None, style="halves", q=None, q_out=None,
                          workspace=None, stream=None) -> None:
    """Keys and values of new tokens into a paged cache, keys (and queries) rotated
    by their positions on the way.

    k, v: bf16/fp32 [T, Hkv, Dh]; positions, slots: int32 [T] (a token with a
    negative slot is skipped, slot s is token s % page_size of page s // page_size);
    k_cache, v_cache: bf16 [pages, page_size, Hkv, Dh], any strides of the first three
    dimensions; inv_freq: fp32 [rot / 2] (None: no rotation); style "halves":
    component j turns with j + rot/2, "pairs": 2j with 2j + 1; q: like k, [T, H, Dh],
    rotated into q_out (bf16; q itself, if bf16)."""
    ldk, ldv = _heads(k, "k"), _heads(v, "v")
    T, Hkv, Dh = k.shape
    if v.shape != k.shape or v.dtype != k.dtype:
        raise ValueError("k and v must be alike")
    shape, sp, st_, sh = _cache(k_cache, v_cache)
    if shape[2] != Hkv or shape[3] != Dh:
        raise ValueError("k_cache must be [pages, page_size, %d, %d], not %s" % (Hkv, Dh, tuple(shape)))
    H, ldq, ldqo = 0, 0, 0
    if q is not None:
        ldq, ldqo = _heads(q, "q"), _heads(q_out, "q_out", _BF16)
        qs = q.shape
        H = qs[1]
        if qs != (T, H, Dh) or q_out.shape != qs or q.dtype is not k.dtype:
            raise ValueError("q and q_out must be [T, H, Dh], q of k's type")
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    ws, _ = _ws(workspace)
    st = _lib().wst_cache_append_bf16(
        T, H, Hkv, Dh, rot, _STYLES[style] if isinstance(style, str) else int(style), _w._ptr(q), ldq, k.data_ptr(), ldk,
        v.data_ptr(), ldv, _type(k, "k"), None if positions is None else _dense(positions, "positions", _I32, (T,)),
        None if not rot else _dense(inv_freq, "inv_freq", _F32, (rot // 2,)), _dense(slots, "slots", _I32, (T,)),
        _w._ptr(q_out) if q is not None else None, ldqo, k_cache.data_ptr(), v_cache.data_ptr(), shape[0], shape[1],
        sp, st_, sh, ws, _stream(stream, k))
    _w._check(st, "wst_cache_append_bf16")


# ----------------------------------------------------------------------------
# attention
# ----------------------------------------------------------------------------
def wst_tree_attention_workspace_size() -> int:
    return int(_lib().wst_tree_attention_workspace_size())


def tree_attention_workspace(device=None, stream=None) -> torch.Tensor:
    """A zero-filled workspace with which wst_tree_attention_bf16 spreads long
    sequences over all SMs; any workspace() works."""
    ws = torch.empty(wst_tree_attention_workspace_size(), dtype=torch.uint8, device=device or "cuda")
    _w.wst_workspace_init(ws, stream)
    return ws


def wst_tree_attention_bf16(Q, q_offsets, context, k_cache, v_cache, page_table, O, mask=None, scale=None, workspace=None,
                            stream=None) -> None:
    """Attention of the new tokens of B sequences over a paged cache that holds them
    already, behind each sequence's context.

    Q: bf16 [T, H, Dh]; q_offsets: device int32 [B+1], the tokens of each sequence;
    context: device int32 [B], its cached tokens before them; k_cache, v_cache: bf16
    [pages, page_size, Hkv, Dh]; page_table: int32 [B, max_pages]; O: bf16/fp32 [T, H,
    Dh]; mask: int32 [T, words], bit d of a row set where the token sees its
    sequence's new token d, or None (those up to itself); scale: 1/sqrt(Dh) if None.
    A token that sees nothing gets zeros; rows behind q_offsets[B] are left as they
    were."""
    ldq, ldo = _heads(Q, "Q", _BF16), _heads(O, "O")
    T, H, Dh = Q.shape
    if O.shape != Q.shape:
        raise ValueError("O must be like Q")
    if not (isinstance(page_table, torch.Tensor) and page_table.dtype is _I32 and page_table.is_cuda and page_table.dim() == 2
            and page_table.stride(1) == 1):
        _need(page_table, "page_table", _I32, (2,))
    B, max_pages = page_table.shape
    shape, sp, st_, sh = _cache(k_cache, v_cache)
    Hkv = shape[2]
    if shape[3] != Dh or Hkv == 0 or H % Hkv:
        raise ValueError("k_cache must be [pages, page_size, Hkv, %d] with Hkv a divisor of %d, not %s" % (Dh, H, tuple(shape)))
    words = ldm = 0
    if mask is not None:
        if not (isinstance(mask, torch.Tensor) and mask.dtype is _I32 and mask.is_cuda and mask.dim() == 2 and mask.stride(1) == 1):
            _need(mask, "mask", _I32, (2,))
        rows, words = mask.shape
        if rows != T or (words < 1 and T > 0):  # (an empty tensor's address is NULL, which means a chain)
            raise ValueError("mask must be [T, words], a word at least")
        ldm = mask.stride(0) if T > 1 else words
    if scale is None:
        scale = 1.0 / math.sqrt(Dh)
    ws, n = _ws(workspace)
    st = _lib().wst_tree_attention_bf16(
        B, T, H, Hkv, Dh, Q.data_ptr(), ldq, _dense(q_offsets, "q_offsets", _I32, (B + 1,)), _dense(context, "context", _I32, (B,)),
        _w._ptr(mask), words, ldm, k_cache.data_ptr(), v_cache.data_ptr(), shape[0], shape[1], sp, st_, sh,
        page_table.data_ptr(), max_pages, page_table.stride(0) if B > 1 else max_pages, scale, O.data_ptr(), ldo, _type(O, "O"), ws, n,
        _stream(stream, Q))
    _w._check(st, "wst_tree_attention_bf16")


# ----------------------------------------------------------------------------
# products with 4-bit weights
# ----------------------------------------------------------------------------
def wst_gemm_w4_workspace_size() -> int:
    return int(_lib().wst_gemm_w4_workspace_size())


def gemm_w4_workspace(device=None, stream=None) -> torch.Tensor:
    """A zero-filled workspace with which the 4-bit products use all SMs; any
    workspace() works."""
    ws = torch.empty(wst_gemm_w4_workspace_size(), dtype=torch.uint8, device=device or "cuda")
    _w.wst_workspace_init(ws, stream)
    return ws


def wst_gemm_w4_tile_rows(M: int, N: int, K: int, groups: int = 0, num_sms: int | None = None) -> int:
    """Rows of a tile (8, 16 or 32: a form of the kernel each) that a product of these
    sizes takes on num_sms SMs (the current device's if None); groups 0: wst_gemm_w4."""
    if num_sms is None:
        num_sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    return int(_lib().wst_gemm_w4_tile_rows(groups, M, N, K, num_sms))


def _w4_operands(A, W, scales, C, group, dims):
    """Checks the operands that both products have; returns their leading dimensions."""
    if A.dtype is not _BF16 or scales.dtype is not _BF16 or W.dtype is not torch.uint8:
        raise TypeError("A and scales must be bfloat16, W uint8")
    lda, ldw, lds, ldc = _rows(A, "A"), _rows(W, "W", dims), _rows(scales, "scales", dims), _rows(C, "C")
    (M, K), N = A.shape, W.shape[-2]
    if W.shape[-1] != -(-K // 2) or group < 1 or tuple(scales.shape) != (*W.shape[:-2], -(-K // group), N) or tuple(C.shape) != (M, N):
        raise ValueError("shape mismatch: A %s W %s scales %s C %s, group %d"
                         % (tuple(A.shape), tuple(W.shape), tuple(scales.shape), tuple(C.shape), group))
    return lda, ldw, lds, ldc


def wst_gemm_w4(A, W, scales, C, group=128, bias=None, epi="none", workspace=None, stream=None) -> None:
    """C = epi(A . w^T (+ bias)), w[n, k] = scales[k // group, n] * (W's 4-bit number - 8).

    A: bf16 [M, K]; W: uint8 [N, ceil(K/2)], two numbers a byte, the even k in the low
    half; scales: bf16 [ceil(K/group), N]; group 32, 64 or 128; C: bf16/fp32 [M, N];
    bias: bf16 [N].  For few rows: every 32 rows read the weights once."""
    lda, ldw, lds, ldc = _w4_operands(A, W, scales, C, group, 2)
    (M, K), N = A.shape, W.shape[0]
    e = _w._epi(epi)
    ws, n = _ws(workspace)
    st = _lib().wst_gemm_w4(
        M, N, K, A.data_ptr(), lda, W.data_ptr(), ldw, scales.data_ptr(), lds, group, _dense(bias, "bias", _BF16, (N,)) if e else None,
        C.data_ptr(), ldc, _type(C, "C"), e, ws, n, _stream(stream, C))
    _w._check(st, "wst_gemm_w4")


def wst_grouped_gemm_w4(A, W, scales, offsets, C, group=128, bias=None, epi="none", workspace=None, stream=None) -> None:
    """Rows [off[g], off[g+1]) of C = epi(rows of A . w[g]^T (+ bias[g])), W [G, N,
    ceil(K/2)] and scales [G, ceil(K/group), N] as in wst_gemm_w4; offsets: device
    int32 [G+1]; bias: bf16 [G, N].  Rows behind offsets[G] are left as they were."""
    lda, ldw, lds, ldc = _w4_operands(A, W, scales, C, group, 3)
    (M, K), (G, N) = A.shape, W.shape[:2]
    off = _dense(offsets, "offsets", _I32, (G + 1,))
    e = _w._epi(epi)
    sbias = 0
    if e:
        _need(bias, "bias", _BF16, (2,))
        if tuple(bias.shape) != (G, N):
            raise ValueError("bias must be [G, N]")
        sbias = bias.stride(0)
    ws, n = _ws(workspace)
    st = _lib().wst_grouped_gemm_w4(
        G, M, N, K, A.data_ptr(), lda, W.data_ptr(), ldw, W.stride(0), scales.data_ptr(), lds, scales.stride(0), group, off,
        _w._ptr(bias) if e else None, sbias, C.data_ptr(), ldc, _type(C, "C"), e, ws, n, _stream(stream, C))
    _w._check(st, "wst_grouped_gemm_w4")
