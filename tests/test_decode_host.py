"""Host-only checks of the decoding-step entry points (no GPU): refusals with the
documented status before anything is enqueued, the binding's own checks, and the
workspace sizes."""
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


APPEND = dict(T=8, H=8, Hkv=2, Dh=128, rot=64, style=0, q=FAKE, ldq=1024, k=FAKE, ldk=256, v=FAKE, ldv=256, xt=1, pos=FAKE, inv=FAKE,
              slots=FAKE, qo=FAKE + 4096, ldqo=1024, kc=FAKE, vc=FAKE, pages=4, page=16, ps=4096, ts=256, hs=128, ws=FAKE, st=None)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INVALID), (dict(Hkv=0), INVALID), (dict(H=0), INVALID), (dict(Dh=0), INVALID), (dict(rot=-16), INVALID),
    (dict(rot=144), INVALID), (dict(Dh=120, rot=16), UNSUPPORTED), (dict(rot=24), UNSUPPORTED),
    (dict(Dh=272, ldq=8 * 272, ldk=544, ldv=544, ldqo=8 * 272, hs=272), UNSUPPORTED), (dict(T=2 ** 31 - 1), UNSUPPORTED),
    (dict(Hkv=2 ** 26), UNSUPPORTED), (dict(style=2), INVALID), (dict(style=-1), INVALID), (dict(xt=2), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(slots=None), INVALID), (dict(qo=None), INVALID), (dict(pos=None), INVALID), (dict(inv=None), INVALID),
    (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(ws=None), INVALID), (dict(pages=0), INVALID), (dict(page=0), INVALID),
    (dict(pages=2 ** 20, page=2 ** 11), UNSUPPORTED), (dict(ps=-8), INVALID), (dict(ts=-8), INVALID), (dict(hs=-8), INVALID),
    (dict(hs=120), INVALID), (dict(ldk=248), INVALID), (dict(ldv=248), INVALID), (dict(ldq=1016), INVALID), (dict(ldqo=1016), INVALID),
    (dict(qo=FAKE, xt=0), INVALID), (dict(qo=FAKE, ldqo=1032), INVALID), (dict(ldk=260), ALIGN), (dict(ldq=1028), ALIGN),
    (dict(ldqo=1028), ALIGN), (dict(ps=4100), ALIGN), (dict(ts=260), ALIGN), (dict(hs=132), ALIGN), (dict(kc=FAKE + 8), ALIGN),
    (dict(k=FAKE + 8), ALIGN), (dict(q=FAKE + 2), ALIGN), (dict(pos=FAKE + 2), ALIGN), (dict(inv=FAKE + 1), ALIGN),
    (dict(slots=FAKE + 2), ALIGN), (dict(ws=FAKE + 8), ALIGN),
    (dict(), INVALID),  # not device memory (no GPU here)
])
def test_append_rejects(lib, change, code):
    assert call(lib, "wst_cache_append_bf16", APPEND, **change) == code
    assert lib.wst_last_error().decode() != ""


ATTEND = dict(B=2, T=8, H=8, Hkv=2, Dh=128, Q=FAKE, ldq=1024, off=FAKE, ctx=FAKE, mask=FAKE, words=1, ldm=1, kc=FAKE, vc=FAKE, pages=4,
              page=16, ps=4096, ts=256, hs=128, table=FAKE, max_pages=2, ldt=2, scale=0.1, O=FAKE, ldo=1024, ot=1, ws=FAKE, n=256, st=None)


@pytest.mark.parametrize("change,code", [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(Hkv=0), INVALID), (dict(H=0), INVALID), (dict(H=7), INVALID), (dict(Dh=0), INVALID),
    (dict(Dh=96), UNSUPPORTED), (dict(Dh=256), UNSUPPORTED), (dict(H=258, ldq=258 * 128, ldo=258 * 128), UNSUPPORTED),
    (dict(page=4), UNSUPPORTED), (dict(page=24), UNSUPPORTED), (dict(page=192), UNSUPPORTED), (dict(page=0), INVALID),
    (dict(pages=0), INVALID), (dict(pages=2 ** 28), UNSUPPORTED), (dict(ps=0), INVALID), (dict(ts=0), INVALID), (dict(hs=0), INVALID),
    (dict(ps=-8), INVALID), (dict(ts=260), ALIGN), (dict(max_pages=0), INVALID), (dict(max_pages=2 ** 27, ldt=2 ** 27), UNSUPPORTED),
    (dict(T=2 ** 30 + 1), UNSUPPORTED), (dict(B=2 ** 29 + 1), UNSUPPORTED), (dict(ot=2), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(scale=3e38), INVALID), (dict(Q=None), INVALID), (dict(O=None), INVALID), (dict(off=None), INVALID), (dict(ctx=None), INVALID),
    (dict(table=None), INVALID), (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(ws=None), INVALID), (dict(ldq=1016), INVALID),
    (dict(ldo=1016), INVALID), (dict(ldt=1), INVALID), (dict(words=0), INVALID), (dict(words=3, ldm=2), INVALID), (dict(Q=FAKE + 8), ALIGN),
    (dict(O=FAKE + 8), ALIGN), (dict(ldq=1028), ALIGN), (dict(ldo=1028), ALIGN), (dict(ldo=1026, ot=0), ALIGN), (dict(off=FAKE + 2), ALIGN),
    (dict(ctx=FAKE + 2), ALIGN), (dict(mask=FAKE + 2), ALIGN), (dict(table=FAKE + 2), ALIGN), (dict(ws=FAKE + 8), ALIGN),
    (dict(n=255), INVALID), (dict(), INVALID)])
def test_attention_rejects(lib, change, code):
    assert call(lib, "wst_tree_attention_bf16", ATTEND, **change) == code
    assert lib.wst_last_error().decode() != ""


GEMM4 = dict(M=8, N=128, K=256, A=FAKE, lda=256, W=FAKE, ldw=128, s=FAKE, lds=128, group=128, bias=None, C=FAKE, ldc=128, ct=1, epi=0,
             ws=FAKE, n=256, st=None)


@pytest.mark.parametrize("change,code", [
    (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(M=2 ** 31 - 1), UNSUPPORTED),
    (dict(K=2 ** 31 - 1, lda=2 ** 31, ldw=2 ** 30), UNSUPPORTED), (dict(group=16), UNSUPPORTED), (dict(group=0), UNSUPPORTED),
    (dict(group=256), UNSUPPORTED), (dict(ct=2), INVALID), (dict(epi=4), INVALID), (dict(epi=1), INVALID), (dict(A=None), INVALID),
    (dict(C=None), INVALID), (dict(W=None), INVALID), (dict(s=None), INVALID), (dict(ws=None), INVALID), (dict(lda=248), INVALID),
    (dict(ldw=112), INVALID), (dict(K=257, lda=264), INVALID), (dict(lds=120), INVALID), (dict(ldc=120), INVALID), (dict(lda=260), ALIGN),
    (dict(ldw=136), ALIGN), (dict(lds=132), ALIGN), (dict(ldc=132), ALIGN), (dict(ldc=130, ct=0), ALIGN), (dict(A=FAKE + 8), ALIGN),
    (dict(W=FAKE + 8), ALIGN), (dict(s=FAKE + 8), ALIGN), (dict(C=FAKE + 8), ALIGN), (dict(epi=1, bias=FAKE + 1), ALIGN),
    (dict(ws=FAKE + 8), ALIGN), (dict(n=255), INVALID), (dict(), INVALID)])
def test_gemm_rejects(lib, change, code):
    assert call(lib, "wst_gemm_w4", GEMM4, **change) == code
    assert lib.wst_last_error().decode() != ""


GROUP4 = dict(G=4, M=8, N=128, K=256, A=FAKE, lda=256, W=FAKE, ldw=128, stW=128 * 128, s=FAKE, lds=128, stS=256, group=128, off=FAKE,
              bias=None, stBias=0, C=FAKE, ldc=128, ct=1, epi=0, ws=FAKE, n=256, st=None)


@pytest.mark.parametrize("change,code", [
    (dict(G=0), INVALID), (dict(M=-1), INVALID), (dict(off=None), INVALID), (dict(off=FAKE + 2), ALIGN), (dict(stW=-16), INVALID),
    (dict(stW=8), ALIGN), (dict(stS=-8), INVALID), (dict(stS=4), ALIGN), (dict(epi=1, bias=FAKE, stBias=-1), INVALID), (dict(ct=5), INVALID),
    (dict(G=2 ** 31 - 1000), UNSUPPORTED),
    (dict(G=2 ** 24, N=2 ** 20, lds=2 ** 20, ldc=2 ** 20), INVALID),  # (too large too, which only the device's sizes decide)
    (dict(), INVALID)])
def test_grouped_gemm_rejects(lib, change, code):
    assert call(lib, "wst_grouped_gemm_w4", GROUP4, **change) == code


def test_nothing_to_do_is_fine(lib):
    # no tokens, no rows: nothing is enqueued, and NULL arrays are not looked at
    assert call(lib, "wst_cache_append_bf16", APPEND, T=0, k=None, v=None, slots=None, pos=None) == wst.WST_OK
    assert call(lib, "wst_tree_attention_bf16", ATTEND, T=0, Q=None, O=None, off=None, ctx=None, table=None) == wst.WST_OK
    assert call(lib, "wst_tree_attention_bf16", ATTEND, B=0, max_pages=0, Q=None, O=None, off=None, ctx=None, table=None) == wst.WST_OK
    assert call(lib, "wst_gemm_w4", GEMM4, M=0, A=None, C=None) == wst.WST_OK
    assert call(lib, "wst_grouped_gemm_w4", GROUP4, M=0, A=None, C=None) == wst.WST_OK


def test_workspace_sizes():
    # two slots of 128 x 128 sums with their maxima and sums for each of 160 blocks; pieces of products
    assert 20 << 20 < wst.wst_tree_attention_workspace_size() < 24 << 20
    assert 256 < wst.wst_gemm_w4_workspace_size() < 32 << 20
    assert wst.wst_tree_attention_workspace_size() % 16 == 0 and wst.wst_gemm_w4_workspace_size() % 16 == 0


def test_binding_checks_its_tensors():
    x, i = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    c = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        wst.wst_cache_append_bf16(x, x, i, i, c, c)                      # not CUDA tensors
    with pytest.raises(TypeError):
        wst.wst_cache_append_bf16([1.0], x, i, i, c, c)
    with pytest.raises(ValueError):
        wst.wst_tree_attention_bf16(x, i, i, c, c, i, x)
    with pytest.raises(TypeError):
        wst.wst_gemm_w4(x[0], i, x[0], x[0])
    with pytest.raises(ValueError):
        wst.wst_gemm_w4(x[0], torch.zeros(8, 32, dtype=torch.uint8), x[0], x[0])
    for name in wst.decode.__all__:
        assert hasattr(wst, name) and name in wst.__all__


def test_every_function_has_its_argument_types(lib):
    for name in [n for n in wst.decode.__all__ if n.startswith("wst_")]:
        fn = getattr(lib, name)
        assert fn.argtypes is not None and fn.restype in (ctypes.c_int, ctypes.c_size_t)
