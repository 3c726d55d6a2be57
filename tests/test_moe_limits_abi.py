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


@pytest.mark.parametrize("fp8", [False, True])
def test_block_norm_columns_of_one_buffer_that_meet_are_refused(L, fp8):
    """Rows of 128 bytes, 384 apart: h_out 64 bytes into x's columns, or reaching into the next
    row's, or codes among them."""
    import ctypes

    f = L.sq_block_norm_quant_per_token_fp8 if fp8 else L.sq_block_norm_quant_per_token
    X, RES, H, Q = 0x1000000, 0x2000000, 0x3000000, 0x4000000
    ok = dict(x=X, ldx=192, R=8, dtype=1, M=8, K=64, post_norm=1, pre_norm=1, post_eps=1e-5, pre_eps=1e-5,
              residual=RES, ld_res=192, residual_scale=1.0, h_out=H, ld_h=192, Xq=Q, x_scale=0x5000000)
    for bad in (dict(h_out=X + 64), dict(h_out=X + 320), dict(h_out=X - 64), dict(h_out=X + 384 * 3 + 112),
                dict(h_out=RES + 112), dict(h_out=RES + 272), dict(h_out=X, token_row=0x6000000,
                                                                  weights=0x7000000, top_k=1),
                dict(h_out=X + 128, ld_h=200), dict(Xq=X + 128), dict(Xq=H + 256)):
        a = sq.BlockNormArgs()
        for k, v in dict(ok, **bad).items():
            setattr(a, k, v)
        assert f(ctypes.byref(a), None) == 1, bad
