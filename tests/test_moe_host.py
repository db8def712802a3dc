"""Host-only checks of the mixture-of-experts entry points (no GPU): refusals with
the documented status before anything is enqueued, the binding's own checks, and
the workspace sizes."""
import ctypes

import pytest
import torch

import warp_specialized_tensor_gb300 as wst

INVALID, ALIGN, UNSUPPORTED = wst.WST_ERR_INVALID_ARG, wst.WST_ERR_ALIGNMENT, wst.WST_ERR_UNSUPPORTED
FAKE = 0x10000  # 16-byte aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    return wst.load_library()


def call(lib, name, base, **change):
    a = dict(base, **change)
    return getattr(lib, name)(*a.values())


ROUTE = dict(T=8, E=64, k=4, logits=FAKE, ld=64, type=0, score=1, bias=None, groups=8, top_groups=4, best=2, renorm=1, scale=1.0,
             experts=FAKE, weights=FAKE, st=None)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(k=65), INVALID), (dict(E=1025, ld=1025), UNSUPPORTED),
    (dict(k=17), UNSUPPORTED), (dict(ld=63), INVALID), (dict(type=2), INVALID), (dict(score=2), INVALID), (dict(groups=0), INVALID),
    (dict(groups=7), INVALID), (dict(groups=64), UNSUPPORTED), (dict(top_groups=9), INVALID), (dict(top_groups=0), INVALID),
    (dict(best=3), INVALID), (dict(best=0), INVALID), (dict(k=9, top_groups=1), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(logits=None), INVALID), (dict(experts=None), INVALID), (dict(weights=None), INVALID),
    (dict(logits=FAKE + 2), ALIGN), (dict(bias=FAKE + 2), ALIGN), (dict(T=2 ** 30), INVALID),
    (dict(), INVALID),  # not device memory (no GPU here)
])
def test_route_rejects(lib, change, code):
    assert call(lib, "wst_moe_route", ROUTE, **change) == code
    assert lib.wst_last_error().decode() != ""


BWD = dict(T=8, E=64, k=4, logits=FAKE, ld=64, type=1, score=0, renorm=1, scale=1.0, experts=FAKE, dw=FAKE, dx=FAKE, ldd=64, st=None)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INVALID), (dict(k=65), INVALID), (dict(E=2000, ld=2000, ldd=2000), UNSUPPORTED), (dict(ldd=63), INVALID),
    (dict(ld=63), INVALID), (dict(dw=None), INVALID), (dict(dx=None), INVALID), (dict(dx=FAKE + 1), ALIGN),
    (dict(experts=FAKE + 2), ALIGN), (dict(score=-1), INVALID), (dict(), INVALID)])
def test_route_backward_rejects(lib, change, code):
    assert call(lib, "wst_moe_route_backward", BWD, **change) == code


PLAN = dict(T=8, k=4, experts=FAKE, E=64, offsets=FAKE, pair=FAKE, token=FAKE, pos=FAKE, ws=FAKE, n=1 << 20, st=None)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(E=0), INVALID), (dict(E=1025), UNSUPPORTED), (dict(T=2 ** 30), INVALID),
    (dict(offsets=None), INVALID), (dict(pos=None), INVALID), (dict(ws=None), INVALID), (dict(n=255), INVALID),
    (dict(T=100000, n=256), INVALID), (dict(ws=FAKE + 8), ALIGN), (dict(pair=FAKE + 2), ALIGN), (dict(), INVALID)])
def test_plan_rejects(lib, change, code):
    assert call(lib, "wst_moe_plan", PLAN, **change) == code


def test_plan_workspace():
    assert wst.wst_moe_plan_workspace_size(0, 8) == 256 and wst.wst_moe_plan_workspace_size(2048, 8) == 256
    big = wst.wst_moe_plan_workspace_size(1 << 20, 1024)
    assert 256 < big <= 256 + 128 * 1024 * 4
    assert wst.wst_moe_plan_workspace_size(-1, 8) == 0 and wst.wst_moe_plan_workspace_size(8, 0) == 0
    # never less for more pairs, so a workspace serves every smaller call
    sizes = [wst.wst_moe_plan_workspace_size(p, 64) for p in (1, 2048, 2049, 3000, 50000, 131071, 131072, 131073, 10 ** 6, 10 ** 8)]
    assert sizes == sorted(sizes) and sizes[-1] == 256 + 128 * 64 * 4


COMB = dict(T=8, k=4, N=64, y=FAKE, ldy=64, yt=1, rows=32, pos=FAKE, w=None, out=FAKE, ldo=64, ot=1, ws=FAKE, st=None)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(k=33), UNSUPPORTED), (dict(N=0), INVALID), (dict(rows=-1), INVALID),
    (dict(ldy=63), INVALID), (dict(ldo=60), INVALID), (dict(ldy=68), ALIGN), (dict(y=FAKE + 8), ALIGN), (dict(ot=3), INVALID),
    (dict(y=None), INVALID), (dict(pos=None), INVALID), (dict(ws=None), INVALID), (dict(w=FAKE + 2), ALIGN), (dict(), INVALID)])
def test_combine_rejects(lib, change, code):
    assert call(lib, "wst_moe_combine", COMB, **change) == code


CBWD = dict(T=8, k=4, N=64, dout=FAKE, ldo=64, ot=1, y=FAKE, ldy=64, yt=1, rows=32, pos=FAKE, w=None, dy=FAKE, lddy=64, dw=FAKE,
            ws=FAKE, st=None)


@pytest.mark.parametrize("change,code", [
    (dict(dy=None, dw=None), INVALID), (dict(y=None), INVALID), (dict(dout=None), INVALID), (dict(lddy=32), INVALID),
    (dict(dw=FAKE + 1), ALIGN), (dict(dy=FAKE + 4), ALIGN), (dict(k=33), UNSUPPORTED), (dict(yt=7), INVALID), (dict(), INVALID)])
def test_combine_backward_rejects(lib, change, code):
    assert call(lib, "wst_moe_combine_backward", CBWD, **change) == code


QUANT = dict(mode=0, batch=1, M=64, K=256, x=FAKE, ldx=256, sx=0, xt=1, q=FAKE, ldq=256, sq=0, qt=0, s=FAKE, lds=64, ss=0, pow2=0, st=None)


@pytest.mark.parametrize("change,code", [
    (dict(mode=4), INVALID), (dict(mode=-1), INVALID), (dict(batch=0), INVALID), (dict(batch=65536), INVALID), (dict(M=-1), INVALID),
    (dict(K=0), INVALID), (dict(xt=2), INVALID), (dict(qt=2), INVALID), (dict(ldx=255), INVALID), (dict(ldq=240), INVALID),
    (dict(lds=63), INVALID), (dict(ldx=260), ALIGN), (dict(ldq=264), ALIGN), (dict(q=FAKE + 8), ALIGN), (dict(x=None), INVALID),
    (dict(mode=1, ldq=48), INVALID), (dict(mode=2, lds=1), INVALID), (dict(batch=2), INVALID),
    (dict(batch=2, sx=64 * 256, sq=64 * 256 + 8, ss=128), ALIGN), (dict(M=65535 * 128 + 1, lds=65535 * 128 + 1), UNSUPPORTED),
    (dict(), INVALID)])
def test_quantize_rejects(lib, change, code):
    assert call(lib, "wst_quantize_fp8", QUANT, **change) == code


DISP = dict(M=64, K=256, copies=2, x=FAKE, ldx=256, xt=1, pos=FAKE, rows=128, q=FAKE, ldq=256, qt=0, s=FAKE, lds=128, pow2=0, ws=FAKE,
            st=None)


@pytest.mark.parametrize("change,code", [
    (dict(copies=0), INVALID), (dict(rows=-1), INVALID), (dict(pos=None), INVALID), (dict(lds=127), INVALID), (dict(ws=None), INVALID),
    (dict(pos=FAKE + 2), ALIGN), (dict(), INVALID)])
def test_quantize_dispatch_rejects(lib, change, code):
    assert call(lib, "wst_quantize_fp8_dispatch", DISP, **change) == code


GEMM8 = dict(M=64, N=128, K=256, A=FAKE, lda=256, at=0, sa=FAKE, ldsa=64, B=FAKE, ldb=256, bt=0, sb=FAKE, ldsb=2, scaling=2, bias=None,
             C=FAKE, ldc=128, ct=1, epi=0, ws=FAKE, n=256, st=None)


@pytest.mark.parametrize("change,code", [
    (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(at=2), INVALID), (dict(ct=2), INVALID), (dict(epi=4), INVALID),
    (dict(epi=1), INVALID), (dict(scaling=1), INVALID), (dict(scaling=3), INVALID), (dict(ws=None), INVALID), (dict(n=255), INVALID),
    (dict(lda=240), INVALID), (dict(ldsa=63), INVALID), (dict(ldsb=1), INVALID), (dict(scaling=0, ldsb=127), INVALID),
    (dict(ldc=120), INVALID), (dict(lda=264), ALIGN), (dict(A=FAKE + 8), ALIGN), (dict(sa=FAKE + 2), ALIGN), (dict(ldc=132), ALIGN),
    (dict(sb=None), INVALID), (dict(), INVALID)])
def test_gemm_fp8_rejects(lib, change, code):
    assert call(lib, "wst_gemm_fp8", GEMM8, **change) == code


GROUP8 = dict(G=4, M=64, N=128, K=256, A=FAKE, lda=256, at=0, sa=FAKE, ldsa=64, B=FAKE, ldb=256, stB=128 * 256, bt=0, sb=FAKE, ldsb=2,
              stS=2, scaling=2, off=FAKE, bias=None, stBias=0, C=FAKE, ldc=128, ct=1, epi=0, ws=FAKE, n=256, st=None)


@pytest.mark.parametrize("change,code", [
    (dict(G=0), INVALID), (dict(off=None), INVALID), (dict(off=FAKE + 2), ALIGN), (dict(stB=-16), INVALID), (dict(stB=8), ALIGN),
    (dict(stS=-1), INVALID), (dict(), INVALID)])
def test_grouped_gemm_fp8_rejects(lib, change, code):
    assert call(lib, "wst_grouped_gemm_fp8", GROUP8, **change) == code


WGRAD = dict(G=4, M=64, N=128, K=256, dC=FAKE, lddc=128, A=FAKE, lda=256, off=FAKE, dB=FAKE, lddb=256, stB=128 * 256, t=0, acc=0, ws=FAKE,
             st=None)


@pytest.mark.parametrize("change,code", [
    (dict(G=0), INVALID), (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(t=2), INVALID), (dict(lddc=120), INVALID),
    (dict(lddb=248), INVALID), (dict(stB=100), INVALID), (dict(dB=None), INVALID), (dict(dC=None), INVALID), (dict(ws=None), INVALID),
    (dict(lda=260), ALIGN), (dict(dB=FAKE + 8), ALIGN), (dict(off=FAKE + 2), ALIGN), (dict(stB=128 * 256 + 2), ALIGN), (dict(), INVALID)])
def test_wgrad_rejects(lib, change, code):
    assert call(lib, "wst_grouped_gemm_wgrad_bf16", WGRAD, **change) == code


def test_nothing_to_do_is_fine(lib):
    # no tokens, no rows: nothing is enqueued, and NULL arrays are not looked at
    assert call(lib, "wst_moe_route", ROUTE, T=0, logits=None, experts=None, weights=None) == wst.WST_OK
    assert call(lib, "wst_moe_route_backward", BWD, T=0, logits=None) == wst.WST_OK
    assert call(lib, "wst_quantize_fp8", QUANT, M=0, x=None, q=None, s=None, lds=0) == wst.WST_OK
    assert call(lib, "wst_gemm_fp8", GEMM8, M=0, A=None, C=None) == wst.WST_OK
    assert call(lib, "wst_moe_combine", COMB, T=0, out=None, pos=None) == wst.WST_OK


def test_binding_checks_its_tensors():
    x = torch.zeros(4, 8)
    i = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        wst.wst_moe_route(x, i, torch.zeros(4, 2))                     # not CUDA tensors
    with pytest.raises(TypeError):
        wst.wst_moe_route([1.0], i, torch.zeros(4, 2))
    with pytest.raises(ValueError):
        wst.wst_moe_combine(x, i, x)
    with pytest.raises(ValueError):
        wst.wst_quantize_fp8(x, x, x)
    for name in wst.moe.__all__:
        assert hasattr(wst, name) and name in wst.__all__


def test_every_function_has_its_argument_types(lib):
    for name in [n for n in wst.moe.__all__ if n.startswith("wst_")]:
        fn = getattr(lib, name)
        assert fn.argtypes is not None and fn.restype in (ctypes.c_int, ctypes.c_size_t)


def test_flag_values_equal_no_count_and_no_sum(lib):
    # A workspace may hold the plan's counts or fp32 sums where another operation
    # keeps its ready flags: the flags' values are NaNs that arithmetic does not return.
    import numpy as np
    fresh = getattr(lib, "_ZN3wst15next_flag_epochEv")
    fresh.restype = ctypes.c_uint32
    v = np.array([fresh() for _ in range(100000)], dtype=np.uint32)
    assert len(set(v.tolist())) == v.size
    assert np.isnan(v.view(np.float32)).all() and not np.isin(v, [0x7fffffff, 0xffffffff]).any()


@pytest.mark.parametrize("k", [1, 2, 4])
def test_combine_rejects_what_32_bits_do_not_hold(lib, k):
    # A thread's next columns are at most 128 threads x 8 vectors x 8 columns on, a
    # block's tokens at most 4: beyond that an index would turn negative.  (INVALID:
    # past the check of the sizes, not device memory.)
    widest = 2 ** 31 - 1 - 8 * 128 * 8
    ld = 2 ** 31
    for N, T, code in ((widest, 8, INVALID), (widest + 1, 8, UNSUPPORTED), (2 ** 31 - 1 - 8 * 128 * 4, 8, UNSUPPORTED),
                       (64, 2 ** 31 - 1, UNSUPPORTED), (64, 2 ** 31 - 1025, INVALID)):
        assert call(lib, "wst_moe_combine", COMB, N=N, T=T, k=k, ldy=ld, ldo=ld) == code
        assert call(lib, "wst_moe_combine_backward", CBWD, N=N, T=T, k=k, ldy=ld, ldo=ld, lddy=ld) == code


def test_route_rejects_more_tokens_than_32_bits_hold(lib):
    for T, code in ((2 ** 31 - 1, UNSUPPORTED), (2 ** 31 - 1024, UNSUPPORTED), (2 ** 31 - 1025, INVALID)):
        assert call(lib, "wst_moe_route", ROUTE, T=T) == code                # (too many pairs, below)
        assert call(lib, "wst_moe_route_backward", BWD, T=T, k=1) == code    # (not device memory, below)


def test_dispatch_to_no_rows_needs_no_arrays(lib):
    assert call(lib, "wst_quantize_fp8_dispatch", DISP, rows=128, q=None) == INVALID and b"NULL" in lib.wst_last_error()
    assert call(lib, "wst_quantize_fp8_dispatch", DISP, rows=0, q=None, s=None) == INVALID
    assert b"NULL" not in lib.wst_last_error()                       # (x is not device memory here)


def test_combine_backward_to_no_rows(lib):
    for rows, said in ((32, True), (0, False)):
        assert call(lib, "wst_moe_combine_backward", CBWD, rows=rows, dy=None, dw=None, y=None) == INVALID
        assert (b"neither" in lib.wst_last_error()) == said          # (else: not device memory here)


def test_one_group_has_no_stride(lib):
    # (what is left to refuse is that nothing here is device memory)
    for G, code in ((4, ALIGN), (1, INVALID)):
        assert call(lib, "wst_grouped_gemm_fp8", GROUP8, G=G, stB=100) == code
