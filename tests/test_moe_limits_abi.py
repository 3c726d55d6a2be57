"""How far the expert-layer calls reach, read from their refusals: no GPU needed (a K that is not a
multiple of 16 is refused after the sizes, so nothing is ever launched)."""
import pytest

from w8a8_int8_quantized_norm_b200 import build as sqbuild
from w8a8_int8_quantized_norm_b200 import sq

from test_lib_abi import A16

UNSUPPORTED, ALIGNMENT = 2, 3


@pytest.fixture(scope="module")
def L():
    sqbuild.build()
    return sq.lib()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("R,E,N,path,want", [
    # 2^30 tiles of up to 256 (decode: 32) rows and 256 (128) columns are the limit
    (2_000_000, 8, 1 << 20, 0, ALIGNMENT), (2_000_000, 8, 1 << 20, 1, ALIGNMENT),
    (2_000_000, 8, 1 << 20, 2, ALIGNMENT), (1 << 24, 1, 1 << 20, 1, ALIGNMENT),
    (1 << 24, 1, 1 << 20, 2, UNSUPPORTED), (1 << 30, 1, 1 << 22, 1, UNSUPPORTED),
    (1 << 30, 1, 1 << 22, 0, UNSUPPORTED)])
def test_grouped_tiles_in_32_bits(L, R, E, N, path, want, fp8):
    f = L.sq_fp8_gemm_grouped if fp8 else L.sq_w8a8_gemm_grouped
    assert f(A16, R, A16, A16, A16, A16, None, R, E, N, 24, 0, A16, N, path, None) == want
