"""Binding of the mixture-of-experts operators around the grouped GEMM: routing,
the plan of the rows, the sum of the experts' rows, 8-bit products with block
scales, and the gradients (``include/wst.h`` has the definitions).

The functions are exported by the package.  They follow its conventions: the
C ABI's names, outputs passed in, sizes and leading dimensions read from the
tensors, the current stream unless one is given.
"""
from __future__ import annotations

import ctypes

import torch

import warp_specialized_tensor_gb300 as _w

__all__ = [
    "SCORE_SOFTMAX", "SCORE_SIGMOID", "E4M3", "E5M2", "FP8_ROWS", "FP8_COLS", "FP8_BLOCKS", "FP8_BLOCKS_T",
    "wst_moe_route", "wst_moe_route_backward", "wst_moe_plan", "wst_moe_plan_workspace_size", "moe_plan_workspace",
    "wst_moe_combine", "wst_moe_combine_backward", "wst_quantize_fp8", "wst_quantize_fp8_dispatch",
    "wst_gemm_fp8", "wst_grouped_gemm_fp8", "wst_gemm_fp8_workspace_size", "gemm_fp8_workspace",
    "wst_grouped_gemm_wgrad_bf16",
]

# enums of include/wst.h
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
E4M3, E5M2 = 0, 1
FP8_ROWS, FP8_COLS, FP8_BLOCKS, FP8_BLOCKS_T = 0, 1, 2, 3
_SCORES = {"softmax": SCORE_SOFTMAX, "sigmoid": SCORE_SIGMOID}
_MODES = {"rows": FP8_ROWS, "cols": FP8_COLS, "blocks": FP8_BLOCKS, "blocks_t": FP8_BLOCKS_T}
_FP8 = {torch.float8_e4m3fn: E4M3, torch.float8_e5m2: E5M2}


def declare(lib) -> None:
    """Argument types of the functions bound here."""
    P, I, L, Z, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_long, ctypes.c_size_t, ctypes.c_float
    for name, res, args in (
            ("wst_moe_route", I, [I, I, I, P, L, I, I, P, I, I, I, I, F, P, P, P]),
            ("wst_moe_route_backward", I, [I, I, I, P, L, I, I, I, F, P, P, P, L, P]),
            ("wst_moe_plan", I, [I, I, P, I, P, P, P, P, P, Z, P]),
            ("wst_moe_plan_workspace_size", Z, [I, I]),
            ("wst_moe_combine", I, [I, I, I, P, L, I, I, P, P, P, L, I, P, P]),
            ("wst_moe_combine_backward", I, [I, I, I, P, L, I, P, L, I, I, P, P, P, L, P, P, P]),
            ("wst_quantize_fp8", I, [I, I, I, I, P, L, L, I, P, L, L, I, P, L, L, I, P]),
            ("wst_quantize_fp8_dispatch", I, [I, I, I, P, L, I, P, I, P, L, I, P, L, I, P, P]),
            ("wst_gemm_fp8", I, [I, I, I, P, L, I, P, L, P, L, I, P, L, I, P, P, L, I, I, P, Z, P]),
            ("wst_grouped_gemm_fp8", I, [I, I, I, I, P, L, I, P, L, P, L, L, I, P, L, L, I, P, P, L, P, L, I, I, P, Z, P]),
            ("wst_gemm_fp8_workspace_size", Z, []),
            ("wst_grouped_gemm_wgrad_bf16", I, [I, I, I, I, P, L, P, L, P, P, L, L, I, I, P, P])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args


# The checks below first ask everything in one expression, which is all a good
# call pays for, and look for what is wrong only when it fails.
_I32, _F32 = torch.int32, torch.float32


def _fp8(t, name) -> int:
    if t.dtype not in _FP8:
        raise TypeError("%s must be float8_e4m3fn or float8_e5m2" % name)
    return _FP8[t.dtype]


def _type(t, name) -> int:
    if t.dtype is _F32:
        return _w.F32
    if t.dtype is torch.bfloat16:
        return _w.BF16
    raise TypeError("%s must be float32 or bfloat16" % name)


def _need(t, name, dtype=None, dims=None):
    """The package's check, for tensors whose last stride means nothing (one column, or no element) too."""
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dim() and (t.shape[-1] == 1 or t.numel() == 0):
        if dtype is not None and t.dtype != dtype:
            raise TypeError("%s must be %s" % (name, dtype))
        if dims is not None and t.dim() not in dims:
            raise ValueError("%s must have %s dimensions" % (name, dims))
        return
    _w._need(t, name, dtype, dims)


def _dense(t, name, dtype, shape):
    """A contiguous CUDA tensor of this type and shape; returns its address."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_cuda and t.shape == shape and t.is_contiguous()):
        _need(t, name, dtype)
        raise ValueError("%s must be a contiguous %s tensor, not %s" % (name, tuple(shape), tuple(t.shape)))
    return t.data_ptr()


def _rows(t, name, dims=2):
    """A CUDA tensor of rows; returns the leading dimension (a lone row has none of its own)."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dim() == dims and t.stride(-1) == 1):
        _need(t, name, None, (dims,))
    if t.shape[-2] > 1:
        return t.stride(-2)
    per = 16 // t.element_size()
    return -(-max(t.shape[-1], 1) // per) * per


def _ws(workspace):
    if workspace is None:
        raise ValueError("workspace is required (see workspace())")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _score(score) -> int:
    return _SCORES[score] if isinstance(score, str) else int(score)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, t) -> int:
    """The handle of `stream`, or of the current stream of t's device."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(t.get_device())
    return _w._stream_handle(stream)


def _lib():
    return _w._lib or _w.load_library()


# ----------------------------------------------------------------------------
# routing
# ----------------------------------------------------------------------------
def _logits(t, name):
    """Logits [T, E]; returns the leading dimension (rows need no alignment of their own)."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dim() == 2 and t.stride(1) == 1):
        _need(t, name, None, (2,))
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def wst_moe_route(logits, experts, weights, score="softmax", bias=None, groups=1, top_groups=None, group_best=1,
                  renorm=True, scale=1.0, stream=None) -> None:
    """The top_k experts of each token and their weights.

    logits: bf16/fp32 [T, E]; experts: int32 [T, top_k] and weights: fp32
    [T, top_k], written; bias: fp32 [E] added to the scores for the choice
    only; groups / top_groups / group_best: keep the top_groups of `groups`
    groups of experts by the sum of their group_best best scores; renorm: the
    weights sum to `scale`.  Experts whose logit is -inf (or the type's lowest
    value) are off; a slot without an expert holds -1 and weight 0."""
    ld = _logits(logits, "logits")
    T, E = logits.shape
    if experts.dim() != 2 or experts.shape[0] != T:
        raise ValueError("experts must be [T, top_k]")
    k = experts.shape[1]
    st = _lib().wst_moe_route(
        T, E, k, logits.data_ptr(), ld, _type(logits, "logits"), _score(score),
        None if bias is None else _dense(bias, "bias", _F32, (E,)), groups, groups if top_groups is None else top_groups,
        group_best, 1 if renorm else 0, scale, _dense(experts, "experts", _I32, (T, k)), _dense(weights, "weights", _F32, (T, k)),
        _stream(stream, logits))
    _w._check(st, "wst_moe_route")


def wst_moe_route_backward(logits, experts, dweights, dlogits, score="softmax", renorm=True, scale=1.0, stream=None) -> None:
    """dlogits = the gradient of wst_moe_route's weights for dweights (fp32
    [T, top_k]), the experts held fixed.  dlogits: like logits; the other
    arguments as in wst_moe_route."""
    ld, ldd = _logits(logits, "logits"), _logits(dlogits, "dlogits")
    T, E = logits.shape
    if dlogits.shape != logits.shape or dlogits.dtype != logits.dtype or experts.dim() != 2 or experts.shape[0] != T:
        raise ValueError("dlogits must be like logits, experts [T, top_k]")
    k = experts.shape[1]
    st = _lib().wst_moe_route_backward(
        T, E, k, logits.data_ptr(), ld, _type(logits, "logits"), _score(score), 1 if renorm else 0, scale,
        _dense(experts, "experts", _I32, (T, k)), _dense(dweights, "dweights", _F32, (T, k)), dlogits.data_ptr(), ldd,
        _stream(stream, logits))
    _w._check(st, "wst_moe_route_backward")


def wst_moe_plan_workspace_size(num_pairs: int, num_experts: int) -> int:
    return int(_lib().wst_moe_plan_workspace_size(num_pairs, num_experts))


def moe_plan_workspace(num_pairs: int, num_experts: int, device=None, stream=None) -> torch.Tensor:
    """A zero-filled workspace for wst_moe_plan with up to num_pairs pairs."""
    n = max(wst_moe_plan_workspace_size(num_pairs, num_experts), _w.wst_workspace_size())
    ws = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
    _w.wst_workspace_init(ws, stream)
    return ws


def wst_moe_plan(experts, num_experts, offsets, row_pair, row_token, position, workspace=None, stream=None) -> None:
    """The rows of the grouped product of a routing table: a stable sort of the
    pairs (token, slot) by expert.

    experts: int32 [T, top_k], -1 for no expert; offsets: int32
    [num_experts + 1], the grouped GEMM's offsets; row_pair, row_token: int32
    [T * top_k], the pair and the token of each row (-1 behind the last row);
    position: int32 [T, top_k], the row of each pair (-1: none)."""
    if experts.dim() != 2:
        raise ValueError("experts must be [T, top_k]")
    T, k = experts.shape
    ws, n = _ws(workspace)
    st = _lib().wst_moe_plan(
        T, k, _dense(experts, "experts", _I32, (T, k)), num_experts, _dense(offsets, "offsets", _I32, (num_experts + 1,)),
        _dense(row_pair, "row_pair", _I32, (T * k,)), _dense(row_token, "row_token", _I32, (T * k,)),
        _dense(position, "position", _I32, (T, k)), ws, n, _stream(stream, experts))
    _w._check(st, "wst_moe_plan")


# ----------------------------------------------------------------------------
# combine
# ----------------------------------------------------------------------------
def wst_moe_combine(y, position, out, weights=None, workspace=None, stream=None) -> None:
    """out[t] = sum_i weights[t, i] * y[position[t, i]].

    y: bf16/fp32 [rows, N]; position: int32 [T, top_k], negative entries add
    nothing; weights: fp32 [T, top_k] or None (all 1); out: bf16/fp32 [T, N]."""
    ldy, ldo = _rows(y, "y"), _rows(out, "out")
    T, N = out.shape
    if y.shape[1] != N or position.dim() != 2 or position.shape[0] != T:
        raise ValueError("shape mismatch: y %s position %s out %s" % (tuple(y.shape), tuple(position.shape), tuple(out.shape)))
    k = position.shape[1]
    at = _dense(position, "position", _I32, (T, k))
    w = None if weights is None else _dense(weights, "weights", _F32, (T, k))
    ws, _ = _ws(workspace)
    st = _lib().wst_moe_combine(
        T, k, N, y.data_ptr(), ldy, _type(y, "y"), y.shape[0], at, w, out.data_ptr(), ldo,
        _type(out, "out"), ws, _stream(stream, out))
    _w._check(st, "wst_moe_combine")


def wst_moe_combine_backward(dout, position, y=None, weights=None, dy=None, dweights=None, workspace=None, stream=None) -> None:
    """Gradients of wst_moe_combine: dy[position[t, i]] = weights[t, i] * dout[t]
    and dweights[t, i] = <dout[t], y[position[t, i]]>; either may be None
    (y is needed for dweights only).  Rows of dy that no pair names are left
    as they were."""
    ldo = _rows(dout, "dout")
    T, N = dout.shape
    if position.dim() != 2 or position.shape[0] != T:
        raise ValueError("position must be [T, top_k]")
    k = position.shape[1]
    at = _dense(position, "position", _I32, (T, k))
    w = None if weights is None else _dense(weights, "weights", _F32, (T, k))
    dw = None if dweights is None else _dense(dweights, "dweights", _F32, (T, k))
    if dw is not None and y is None:
        raise ValueError("dweights needs y")
    rows = y if y is not None else dy
    if rows is None:
        raise ValueError("neither dy nor dweights is asked for")
    ldy = _rows(y, "y") if y is not None else 0
    lddy = _rows(dy, "dy") if dy is not None else 0
    if rows.shape[1] != N or (y is not None and dy is not None and (y.shape != dy.shape or y.dtype != dy.dtype)):
        raise ValueError("y and dy must be alike, with rows of N values")
    ws, _ = _ws(workspace)
    st = _lib().wst_moe_combine_backward(
        T, k, N, dout.data_ptr(), ldo, _type(dout, "dout"), _w._ptr(y), ldy, _type(rows, "y"), rows.shape[0],
        at, w, _w._ptr(dy), lddy, dw, ws, _stream(stream, dout))
    _w._check(st, "wst_moe_combine_backward")


# ----------------------------------------------------------------------------
# 8-bit quantisation
# ----------------------------------------------------------------------------
def wst_quantize_fp8(x, q, scales, mode="rows", pow2=False, stream=None) -> None:
    """x ~ q * scale in 8 bits with one scale for each block of 128.

    x: bf16/fp32 [M, K] or [batch, M, K]; mode "rows": q [M, K], scales
    [ceil(K/128), M]; "cols": q [K, M] (x transposed), scales [ceil(M/128), K];
    "blocks": q [M, K], scales [ceil(M/128), ceil(K/128)]; "blocks_t": both
    transposed.  q: float8_e4m3fn or float8_e5m2; scales: fp32; both with x's
    batch dimension.  pow2: scales are powers of two."""
    m = _MODES[mode] if isinstance(mode, str) else int(mode)
    dims = 3 if x.dim() == 3 else 2
    ldx, ldq, lds = _rows(x, "x", dims), _rows(q, "q", dims), _rows(scales, "scales", dims)
    if scales.dtype is not _F32:
        raise TypeError("scales must be float32")
    M, K = x.shape[-2:]
    mb, kb = -(-M // 128), -(-K // 128)
    want_q = (M, K) if m in (FP8_ROWS, FP8_BLOCKS) else (K, M)
    want_s = {FP8_ROWS: (kb, M), FP8_COLS: (mb, K), FP8_BLOCKS: (mb, kb), FP8_BLOCKS_T: (kb, mb)}[m]
    lead = tuple(x.shape[:-2])
    if tuple(q.shape) != lead + want_q or tuple(scales.shape) != lead + want_s:
        raise ValueError("mode %r: q must be %s and scales %s" % (mode, lead + want_q, lead + want_s))
    batch = lead[0] if lead else 1
    if batch == 0 or (M == 0 and K > 0):  # (strides of an empty tensor mean nothing)
        return
    s = (lambda t: t.stride(0) if t.dim() == 3 else 0)
    st = _lib().wst_quantize_fp8(
        m, batch, M, K, x.data_ptr(), ldx, s(x), _type(x, "x"), q.data_ptr(), ldq, s(q), _fp8(q, "q"), scales.data_ptr(), lds,
        s(scales), 1 if pow2 else 0, _stream(stream, x))
    _w._check(st, "wst_quantize_fp8")


def wst_quantize_fp8_dispatch(x, position, q, scales, pow2=False, workspace=None, stream=None) -> None:
    """Quantises each token's row (mode "rows") and stores it to the rows
    position[t, i] of q [rows, K] and of the scales [ceil(K/128), rows].

    x: bf16/fp32 [T, K]; position: int32 [T, copies], negative entries are
    skipped; rows that no entry names are left as they were."""
    ldx, ldq, lds = _rows(x, "x"), _rows(q, "q"), _rows(scales, "scales")
    T, K = x.shape
    rows = q.shape[0]
    if q.shape[1] != K or tuple(scales.shape) != (-(-K // 128), rows) or scales.dtype != torch.float32:
        raise ValueError("q must be [rows, K] and scales float32 [ceil(K/128), rows]")
    if position.dim() != 2:
        raise ValueError("position must be [T, copies]")
    at = _dense(position, "position", _I32, (T, position.shape[1]))
    ws, _ = _ws(workspace)
    st = _lib().wst_quantize_fp8_dispatch(
        T, K, position.shape[1], x.data_ptr(), ldx, _type(x, "x"), at, rows, q.data_ptr(), ldq, _fp8(q, "q"),
        scales.data_ptr(), lds, 1 if pow2 else 0, ws, _stream(stream, x))
    _w._check(st, "wst_quantize_fp8_dispatch")


# ----------------------------------------------------------------------------
# 8-bit products
# ----------------------------------------------------------------------------
def wst_gemm_fp8_workspace_size() -> int:
    return int(_lib().wst_gemm_fp8_workspace_size())


def gemm_fp8_workspace(device=None, stream=None) -> torch.Tensor:
    """A zero-filled workspace with which the 8-bit products can split their K
    loops (products of few tiles); any workspace() works."""
    ws = torch.empty(wst_gemm_fp8_workspace_size(), dtype=torch.uint8, device=device or "cuda")
    _w.wst_workspace_init(ws, stream)
    return ws


def _fp8_operand(q, scale, name, scaling, dims):
    """Checks an 8-bit operand and its scales; returns (ld, type, ld of the scales)."""
    ld, ty, lds = _rows(q, name, dims), _fp8(q, name), _rows(scale, "the scales of " + name, dims)
    if scale.dtype != torch.float32:
        raise TypeError("the scales of %s must be float32" % name)
    R, K = q.shape[-2:]
    kb = -(-K // 128)
    want = (*q.shape[:-2], kb, R) if scaling == FP8_ROWS else (*q.shape[:-2], -(-R // 128), kb)
    if scale.shape != want:
        raise ValueError("the scales of %s must be %s, not %s" % (name, want, tuple(scale.shape)))
    return ld, ty, lds


def wst_gemm_fp8(A, scaleA, B, scaleB, C, scaling="blocks", bias=None, epi="none", workspace=None, stream=None) -> None:
    """C = epi((A * scaleA) . (B * scaleB)^T (+ bias)) for 8-bit A and B.

    A: float8_e4m3fn/e5m2 [M, K] with scaleA fp32 [ceil(K/128), M]; B: [N, K]
    with scaleB [ceil(N/128), ceil(K/128)] (scaling "blocks") or
    [ceil(K/128), N] ("rows"); C: bf16/fp32 [M, N]; bias: bf16 [N].  workspace:
    gemm_fp8_workspace() lets products of few tiles use all SMs."""
    mode = _MODES[scaling] if isinstance(scaling, str) else int(scaling)
    lda, ta, ldsa = _fp8_operand(A, scaleA, "A", FP8_ROWS, 2)
    ldb, tb, ldsb = _fp8_operand(B, scaleB, "B", mode, 2)
    ldc = _rows(C, "C")
    (M, K), N = A.shape, B.shape[0]
    if B.shape[1] != K or tuple(C.shape) != (M, N):
        raise ValueError("shape mismatch: A %s B %s C %s" % (tuple(A.shape), tuple(B.shape), tuple(C.shape)))
    e = _w._epi(epi)
    if e != _w.EPI_NONE:
        _need(bias, "bias", torch.bfloat16, (1,))
        if bias.numel() != N:
            raise ValueError("bias must be [N]")
    ws, n = _ws(workspace)
    st = _lib().wst_gemm_fp8(
        M, N, K, A.data_ptr(), lda, ta, scaleA.data_ptr(), ldsa, B.data_ptr(), ldb, tb, scaleB.data_ptr(), ldsb, mode,
        _w._ptr(bias) if e else None, C.data_ptr(), ldc, _type(C, "C"), e, ws, n, _stream(stream, C))
    _w._check(st, "wst_gemm_fp8")


def wst_grouped_gemm_fp8(A, scaleA, B, scaleB, offsets, C, scaling="blocks", bias=None, epi="none", workspace=None,
                         stream=None) -> None:
    """Rows [off[g], off[g+1]) of C = epi(rows of A . B[g]^T (+ bias[g])) for 8-bit
    A [M_total, K] and B [G, N, K]; scales as in wst_gemm_fp8, scaleB with a
    group dimension; offsets: device int32 [G+1]; bias: bf16 [G, N].  Rows
    behind offsets[G] are left as they were."""
    mode = _MODES[scaling] if isinstance(scaling, str) else int(scaling)
    lda, ta, ldsa = _fp8_operand(A, scaleA, "A", FP8_ROWS, 2)
    ldb, tb, ldsb = _fp8_operand(B, scaleB, "B", mode, 3)
    ldc = _rows(C, "C")
    (M, K), (G, N, K2) = A.shape, B.shape
    if K2 != K or tuple(C.shape) != (M, N):
        raise ValueError("shape mismatch: A %s B %s C %s" % (tuple(A.shape), tuple(B.shape), tuple(C.shape)))
    off = _dense(offsets, "offsets", _I32, (G + 1,))
    e = _w._epi(epi)
    sbias = 0
    if e != _w.EPI_NONE:
        _need(bias, "bias", torch.bfloat16, (2,))
        if tuple(bias.shape) != (G, N):
            raise ValueError("bias must be [G, N]")
        sbias = bias.stride(0)
    ws, n = _ws(workspace)
    st = _lib().wst_grouped_gemm_fp8(
        G, M, N, K, A.data_ptr(), lda, ta, scaleA.data_ptr(), ldsa, B.data_ptr(), ldb, B.stride(0), tb, scaleB.data_ptr(), ldsb,
        scaleB.stride(0), mode, off, _w._ptr(bias) if e else None, sbias, C.data_ptr(), ldc, _type(C, "C"), e, ws,
        n, _stream(stream, C))
    _w._check(st, "wst_grouped_gemm_fp8")


# ----------------------------------------------------------------------------
# weight gradient of the grouped GEMM
# ----------------------------------------------------------------------------
def wst_grouped_gemm_wgrad_bf16(dC, A, offsets, dB, accumulate=False, workspace=None, stream=None) -> None:
    """dB[g] = dC[rows of g]^T . A[rows of g] (added to dB with accumulate).

    dC: bf16 [M_total, N]; A: bf16 [M_total, K]; offsets: device int32 [G+1];
    dB: bf16/fp32 [G, N, K].  Rows behind offsets[G] belong to no group."""
    if dC.dtype is not torch.bfloat16 or A.dtype is not torch.bfloat16:
        raise TypeError("dC and A must be bfloat16")
    lddc, lda, lddb = _rows(dC, "dC"), _rows(A, "A"), _rows(dB, "dB", 3)
    G, N, K = dB.shape
    if A.shape[0] != dC.shape[0] or dC.shape[1] != N or A.shape[1] != K:
        raise ValueError("shape mismatch: dC %s A %s dB %s" % (tuple(dC.shape), tuple(A.shape), tuple(dB.shape)))
    off = _dense(offsets, "offsets", _I32, (G + 1,))
    ws, _ = _ws(workspace)
    st = _lib().wst_grouped_gemm_wgrad_bf16(
        G, dC.shape[0], N, K, dC.data_ptr(), lddc, A.data_ptr(), lda, off, dB.data_ptr(), lddb, dB.stride(0),
        _type(dB, "dB"), 1 if accumulate else 0, ws, _stream(stream, dB))
    _w._check(st, "wst_grouped_gemm_wgrad_bf16")
