"""Refusals of the expert-layer calls: all made on the host, no GPU needed."""
import ctypes
import re

import pytest
import torch

from w8a8_int8_quantized_norm_b200 import build as sqbuild
from w8a8_int8_quantized_norm_b200 import sq

from test_lib_abi import A8, A16, HEADER

A2 = ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module")
def L():
    sqbuild.build()
    return sq.lib()


def test_constants_match_binding():
    text = open(HEADER).read()
    for name, val in (("SQ_MOE_MAX_EXPERTS", sq.MOE_MAX_EXPERTS), ("SQ_MOE_MAX_TOP_K", sq.MOE_MAX_TOP_K),
                      ("SQ_BLOCK_NORM_MAX_K", sq.BLOCK_NORM_MAX_K)):
        assert re.search(r"#define %s %d\b" % (name, val), text), name
    for name, val in sq.MOE_SCORES.items():
        assert re.search(r"\bSQ_MOE_%s\s*=\s*%d\b" % (name.upper(), val), text)
    # the struct's fields, in the header's order
    body = re.search(r"typedef struct sq_block_norm_args \{(.*?)\} sq_block_norm_args;", text, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    names = [n for d in body.split(";") for n in re.findall(r"(\w+)\s*(?:,|$)", d.strip())]
    assert names == [f for f, _ in sq.BlockNormArgs._fields_]


def test_route_refusals(L):
    ok = dict(x=A16, dt=0, T=1000, E=64, ld=64, k=4, score=0, bias=None, renorm=1, scale=1.0, w=A16,
              e=A16, off=A16, row=A16, tok=A16, ws=A16, wsb=1 << 20)

    def call(**kw):
        a = dict(ok, **kw)
        return L.sq_moe_route(*[a[n] for n in ("x", "dt", "T", "E", "ld", "k", "score", "bias", "renorm",
                                               "scale", "w", "e", "off", "row", "tok", "ws", "wsb")], None)

    for bad in (dict(dt=5), dict(T=-1), dict(E=0), dict(ld=63), dict(k=0), dict(k=65), dict(score=2),
                dict(bias=A16), dict(scale=float("nan")), dict(scale=float("inf")), dict(x=None),
                dict(w=None), dict(e=None), dict(off=None), dict(row=None), dict(tok=None)):
        assert call(**bad) == 1, bad
    for bad in (dict(E=513, ld=513), dict(E=64, k=17), dict(T=1 << 30, k=4)):
        assert call(**bad) == 2, bad
    for bad in (dict(x=A2), dict(w=A2), dict(off=A2), dict(score=1, bias=A2), dict(ws=A2)):
        assert call(**bad) == 3, bad
    assert call(dt=1, x=ctypes.c_void_p(0x10001)) == 3
    need = L.sq_moe_route_workspace_size(1000, 64, 4)
    assert need > 0
    assert call(wsb=need - 1) == 7
    assert call(ws=None) == 7
    assert L.sq_moe_route_workspace_size(1, 64, 4) == 0
    assert L.sq_moe_route_workspace_size(0, 64, 4) == 0
    assert L.sq_moe_route_workspace_size(1000, 513, 4) == 0
    # bounded however many tokens there are
    assert L.sq_moe_route_workspace_size(1 << 27, 512, 16) <= 512 * 4 * 4096


@pytest.mark.parametrize("fp8", [False, True])
def test_grouped_refusals(L, fp8):
    f = L.sq_fp8_gemm_grouped if fp8 else L.sq_w8a8_gemm_grouped
    ok = dict(xq=A16, X=64, wq=A16, xs=A16, ws=A16, off=A16, row=None, R=64, E=8, N=256, K=128, epi=0,
              out=A16, ldo=256, path=0)

    def call(**kw):
        a = dict(ok, **kw)
        return f(*[a[n] for n in ("xq", "X", "wq", "xs", "ws", "off", "row", "R", "E", "N", "K", "epi",
                                  "out", "ldo", "path")], None)

    raw, other = (3, 2) if fp8 else (2, 3)
    for bad in (dict(X=-1), dict(R=-1), dict(E=0), dict(N=-1), dict(K=0), dict(ldo=255), dict(epi=other),
                dict(epi=9), dict(path=3), dict(path=-1), dict(X=63), dict(X=0, row=A16), dict(xq=None),
                dict(wq=None), dict(off=None), dict(out=None), dict(xs=None), dict(ws=None)):
        assert call(**bad) == 1, bad
    for bad in (dict(E=513), dict(X=1 << 31, R=1 << 31), dict(N=1 << 29, ldo=1 << 29)):
        assert call(**bad) == 2, bad
    for bad in (dict(K=120), dict(xq=A8), dict(wq=A8), dict(out=ctypes.c_void_p(0x10001)), dict(xs=A2),
                dict(off=A2), dict(row=A2), dict(epi=raw, out=A2)):
        assert call(**bad) == 3, bad
    assert call(K=sq.MAX_K + 8) == 4
    assert call(R=0) == 0 and call(N=0) == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_block_norm_refusals(L, fp8):
    f = L.sq_block_norm_quant_per_token_fp8 if fp8 else L.sq_block_norm_quant_per_token
    ptr = lambda a: a  # noqa: E731
    X, RES, H, Q = 0x1000000, 0x2000000, 0x3000000, 0x4000000
    ok = dict(x=X, ldx=64, R=8, dtype=1, M=8, K=64, post_norm=1, pre_norm=1, post_eps=1e-5,
              pre_eps=1e-5, residual=RES, ld_res=64, residual_scale=1.0, h_out=H, ld_h=64, Xq=Q,
              x_scale=0x5000000)

    def call(**kw):
        a = sq.BlockNormArgs()
        for k, v in dict(ok, **kw).items():
            setattr(a, k, ptr(v))
        return f(ctypes.byref(a), None)

    assert f(None, None) == 1
    for bad in (dict(dtype=3), dict(M=-1), dict(K=0), dict(post_norm=4), dict(pre_norm=-1),
                dict(post_eps=-1.0), dict(pre_eps=float("nan")), dict(h_out=None, Xq=None),
                dict(x=None), dict(ldx=48), dict(ld_res=48), dict(ld_h=48), dict(x_scale=None),
                dict(token_row=0x6000000, top_k=2), dict(weights=0x6000000, top_k=2), dict(top_k=2),
                dict(token_row=0x6000000, weights=0x7000000),
                dict(token_row=0x6000000, weights=0x7000000, top_k=2, R=-1),
                # h_out over its inputs otherwise than row on row
                dict(h_out=X + 128), dict(h_out=RES + 16), dict(h_out=RES, ld_h=72),
                dict(h_out=X, token_row=0x6000000, weights=0x7000000, top_k=1),
                dict(Xq=X), dict(Xq=RES + 512), dict(Xq=H)):
        assert call(**bad) == 1, bad
    for bad in (dict(K=32784, ldx=32784, ld_res=32784, ld_h=32784),
                dict(token_row=0x6000000, weights=0x7000000, top_k=17)):
        assert call(**bad) == 2, bad
    for bad in (dict(x=X + 8), dict(K=56), dict(ldx=68), dict(residual=RES + 2), dict(h_out=H + 8),
                dict(post_gamma=0x6000004), dict(gate=0x6000008), dict(pre_beta=0x6000004),
                dict(token_gate=0x6000002), dict(Xq=Q + 8), dict(x_scale=0x5000002)):
        assert call(**bad) == 3, bad
    assert call(M=0) == 0


def test_binding_refusals_need_no_gpu():
    x = torch.zeros((4, 64))
    with pytest.raises(ValueError, match="CUDA"):
        sq.moe_route(x, 2)
    with pytest.raises(ValueError, match="CUDA"):
        sq.block_norm_quant_per_token(x)
    codes, w = torch.zeros((4, 64), dtype=torch.int8), torch.zeros((2, 8, 64), dtype=torch.int8)
    with pytest.raises(ValueError, match="CUDA"):
        sq.w8a8_gemm_grouped(codes, w, None, None, torch.zeros(3, dtype=torch.int32))
