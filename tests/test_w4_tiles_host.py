"""What the GPU's tests of the 4-bit products reach, by the rule that chooses a product's form (no GPU)."""
import pytest

import warp_specialized_tensor_gb300 as wst
from test_gpu_w4_tiles import DENSE, GROUPS


@pytest.mark.parametrize("sms", [148, 152, 160])
def test_every_form_is_reached_and_cut(sms):
    forms, cut = set(), set()
    for M, N, K, group, _, _, whole, tile in DENSE:
        assert wst.wst_gemm_w4_tile_rows(M, N, K, num_sms=sms) == tile
        forms.add((tile, group))
        tiles, units = -(-M // tile) * -(-N // 128), -(-K // 256)
        if whole and tiles > sms and units > 1 and tiles * units % sms:
            cut.add(tile)
    groups = set()
    for sizes, behind, N, K, group, _, whole, tile in GROUPS:
        assert wst.wst_gemm_w4_tile_rows(sum(sizes) + behind, N, K, groups=len(sizes), num_sms=sms) == tile
        forms.add((tile, group))
        tiles, units = sum(-(-n // tile) for n in sizes) * -(-N // 128), -(-K // 256)
        if whole and tiles > sms and units > 1 and tiles * units % sms:
            groups.add(tile)
    assert forms == {(t, g) for t in (8, 16, 32) for g in (32, 64, 128)}
    assert cut == groups == {8, 16, 32}


def test_sizes_out_of_range():
    for bad in ((-1, 8, 8), (8, 0, 8), (8, 8, 0), (2 ** 31 - 1, 8, 8)):
        assert wst.wst_gemm_w4_tile_rows(*bad, num_sms=152) == 0
    assert wst.wst_gemm_w4_tile_rows(8, 8, 8, groups=-1, num_sms=152) == 0 and wst.wst_gemm_w4_tile_rows(8, 8, 8, num_sms=0) == 0
    assert wst.wst_gemm_w4_tile_rows(0, 8, 8, num_sms=152) == 8
