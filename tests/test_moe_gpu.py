"""The operators of a layer of experts on the GPU against plain 64-bit references."""
import numpy as np
import pytest
import torch

from w8a8_int8_quantized_norm_b200 import sq

import _moe_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    sq.lib()
    yield
    assert sq.get_device_error() == 0


def _rng(*key):
    return np.random.default_rng([7, *key])


def _cuda_of(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def _np64(t):
    return t.double().cpu().numpy()


# ---------------------------------------------------------------------------
# route
# ---------------------------------------------------------------------------

def _check_route(logits, top_k, bias=None, ld=None, **kw):
    T, E = logits.shape
    x = logits
    if ld is not None:
        x = torch.full((T, ld), 99.0, dtype=logits.dtype, device="cuda")
        x[:, :E] = logits
        x = x[:, :E]
    r = sq.moe_route(x, top_k, bias=bias, **kw)
    kw = dict(kw, bias=None if bias is None else bias.cpu().numpy())
    w, e, off, row, tok, bound = ref.route(_np64(logits), top_k, **kw)
    assert np.array_equal(r.experts.cpu().numpy(), e)
    assert np.array_equal(r.offsets.cpu().numpy(), off)
    assert np.array_equal(r.row_token.cpu().numpy(), row)
    assert np.array_equal(r.token_row.cpu().numpy(), tok)
    g = _np64(r.weights)
    # below fp32's normal range a weight is rounded to a multiple of 2^-149
    assert (np.abs(g - w) <= bound * np.abs(w) + 2.0 ** -126).all()
    return r


@pytest.mark.parametrize("T", [0, 1, 2, 63, 64, 65, 129, 1000, 9473])
@pytest.mark.parametrize("E,k", [(1, 1), (4, 2), (8, 8), (33, 3), (64, 6), (128, 8), (200, 5), (512, 16)])
def test_route_sizes(T, E, k):
    if T > 1000 and E > 128:
        T = 700
    logits = _cuda_of(_rng(T, E, k).standard_normal((T, E)).astype(np.float32))
    _check_route(logits, k)


@pytest.mark.parametrize("score,use_bias,renorm", [("softmax", False, False), ("softmax", False, True),
                                                   ("sigmoid", False, False), ("sigmoid", False, True),
                                                   ("sigmoid", True, True), ("sigmoid", True, False)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_scores(score, use_bias, renorm, dtype):
    rng = _rng(1)
    logits = _cuda_of((rng.standard_normal((333, 48)) * 3).astype(np.float32), dtype)
    bias = _cuda_of(rng.standard_normal(48).astype(np.float32)) if use_bias else None
    _check_route(logits, 6, bias, score=score, renormalize=renorm, scale=2.5, ld=61)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_ties_take_the_lowest_index(score):
    rng = _rng(2)
    logits = rng.integers(-2, 3, (500, 70)).astype(np.float32)
    logits[3] = 0.0
    logits[4, ::2] = -0.0
    logits[4, 1::2] = 0.0
    _check_route(_cuda_of(logits, torch.bfloat16), 9, score=score)
    bias = _cuda_of(np.zeros(70, np.float32))
    if score == "sigmoid":
        _check_route(_cuda_of(logits), 9, bias, score=score)


@pytest.mark.parametrize("score,use_bias", [("softmax", False), ("sigmoid", False), ("sigmoid", True)])
def test_route_masked_and_special_logits(score, use_bias):
    rng = _rng(3)
    logits = rng.standard_normal((130, 40)).astype(np.float32)
    lowest = np.finfo(np.float32).min
    logits[0] = -np.inf                      # nothing left
    logits[1] = np.nan
    logits[2, 1:] = -np.inf                  # one expert left
    logits[3, :37] = -np.inf                 # three of four
    logits[4] = lowest                       # the type's lowest value is an ordinary value
    logits[5, 5:] = lowest
    logits[6, 7] = np.inf
    logits[7, [3, 9]] = np.inf
    logits[8, 4] = np.nan
    logits[9] = np.finfo(np.float32).max
    logits[100:] = -np.inf                   # a padded tail
    bias = None
    if use_bias:
        b = rng.standard_normal(40).astype(np.float32)
        b[2], b[11] = -np.inf, np.nan        # experts taken out of service
        bias = _cuda_of(b)
    for renorm in (False, True):
        _check_route(_cuda_of(logits), 4, bias, score=score, renormalize=renorm)


def test_route_every_token_one_expert_and_all_masked():
    logits = np.zeros((3000, 16), np.float32)
    logits[:, 5] = 1.0
    _check_route(_cuda_of(logits), 1)
    _check_route(_cuda_of(np.full((3000, 16), -np.inf, np.float32)), 3)


# ---------------------------------------------------------------------------
# grouped GEMM
# ---------------------------------------------------------------------------

def _codes(rng, shape, fp8):
    if not fp8:
        return rng.integers(-127, 128, shape).astype(np.int8)
    b = rng.integers(0, 256, shape).astype(np.uint8)
    return np.where((b & 0x7f) == 0x7f, 0x31, b).astype(np.uint8)  # finite codes


def _values(codes, fp8):
    return ref.E4M3[codes] if fp8 else codes.astype(np.float64)


def _check_grouped(counts, N, K, fp8=False, gather=None, path=0, epi="bf16", extra_rows=0, pad=0,
                   seed=0, first=0):
    rng = _rng(11, seed, N, K, len(counts))
    E = len(counts)
    off = first + np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R = int(off[-1]) + extra_rows
    X = gather if gather else max(R, 1)
    xq, wq = _codes(rng, (X, K), fp8), _codes(rng, (E, N, K), fp8)
    xs = rng.uniform(1e-3, 1e-2, X).astype(np.float32)
    ws = rng.uniform(1e-4, 1e-3, (E, N)).astype(np.float32)
    row = rng.integers(0, X, R).astype(np.int32) if gather else np.arange(X, dtype=np.int32)
    raw = "f32" if fp8 else "i32"
    is_raw = epi == "raw"
    want = torch.bfloat16 if not is_raw else torch.float32 if fp8 else torch.int32
    # a canary around and behind the rows
    buf = torch.full((R if gather else X, N + pad), 77, dtype=want, device="cuda")
    out = buf[:, :N]
    gemm = sq.fp8_gemm_grouped if fp8 else sq.w8a8_gemm_grouped
    got = gemm(_cuda_of(xq), _cuda_of(wq), _cuda_of(xs), _cuda_of(ws), _cuda_of(off),
               row_token=_cuda_of(row) if gather else None, epi=raw if is_raw else epi, out=out,
               path_hint=path)
    assert got is out
    a, b = _values(xq, fp8)[row], _values(wq, fp8)
    o = out.double().cpu().numpy() if fp8 or not is_raw else out.cpu().numpy().astype(np.float64)
    live = np.zeros(o.shape[0], bool)
    for e in range(E):
        r0, r1 = off[e], off[e + 1]
        live[r0:r1] = True
        acc = a[r0:r1] @ b[e].T  # below 2^53: exact
        if not fp8:
            if is_raw:
                assert np.array_equal(o[r0:r1], acc)
                continue
            t = acc.astype(np.float32) * xs[row[r0:r1], None] * ws[e][None]
            if epi == "bf16_relu":
                t = np.maximum(t, 0)
            exp = torch.from_numpy(t).to(torch.bfloat16).double().numpy()
            assert np.array_equal(o[r0:r1], exp)
        else:
            # summed in the tensor cores' order: (31 + K / 32) 2^-23 of sum |a b|, and one
            # rounding for each of up to 8 joined K ranges
            bound = (31 + -(-K // 32) + 8) * 2.0 ** -23 * (np.abs(a[r0:r1]) @ np.abs(b[e]).T)
            if not is_raw:
                s = xs[row[r0:r1], None].astype(np.float64) * ws[e][None]
                acc, bound = acc * s, bound * s
                if epi == "bf16_relu":
                    acc = np.maximum(acc, 0)
                bound = bound + 2.0 ** -8 * (np.abs(acc) + bound) + 2.0 ** -23 * np.abs(acc)
            assert (np.abs(o[r0:r1] - acc) <= bound).all()
    full = buf.double().cpu().numpy()
    assert (full[~live] == 77).all() and (full[:, N:] == 77).all()


GROUPS = {
    "one": [1], "pair": [1, 1], "empty_mid": [3, 0, 5], "all_empty": [0, 0, 0, 0],
    "ragged": [17, 1, 0, 33, 64, 2, 0, 130], "big": [300, 0, 700, 129], "tail_empty": [40, 0, 0],
    "many": [1 + (i * 7) % 5 for i in range(70)], "edges": [15, 16, 31, 32, 33, 127, 128, 255, 256, 257],
}


@pytest.mark.parametrize("path", [0, 1, 2])
@pytest.mark.parametrize("fp8", [False, True], ids=["int8", "fp8"])
@pytest.mark.parametrize("groups", list(GROUPS))
def test_grouped_group_sizes(groups, fp8, path):
    _check_grouped(GROUPS[groups], 200, 272, fp8, path=path, extra_rows=5, pad=3)
    _check_grouped(GROUPS[groups], 200, 272, fp8, gather=50, path=path, extra_rows=5)


@pytest.mark.parametrize("path", [1, 2])
@pytest.mark.parametrize("fp8", [False, True], ids=["int8", "fp8"])
@pytest.mark.parametrize("N", [1, 7, 127, 128, 129, 256, 257, 1000])
@pytest.mark.parametrize("K", [16, 48, 128, 144, 1040, 4112])
def test_grouped_shapes(N, K, fp8, path):
    _check_grouped([5, 0, 70, 2], N, K, fp8, gather=33, path=path)


@pytest.mark.parametrize("path", [1, 2])
@pytest.mark.parametrize("fp8", [False, True], ids=["int8", "fp8"])
@pytest.mark.parametrize("gather", [None, 300])
def test_grouped_many_tiles_per_cta(gather, fp8, path):
    """Persistent CTAs run several tiles of different widths one after another."""
    _check_grouped([1040, 300, 0, 17, 1, 600, 33], 4000, 1040, fp8, gather=gather, path=path)


@pytest.mark.parametrize("path", [1, 2])
@pytest.mark.parametrize("epi", ["bf16_relu", "raw"])
@pytest.mark.parametrize("fp8", [False, True], ids=["int8", "fp8"])
def test_grouped_epilogues(epi, fp8, path):
    _check_grouped([5, 0, 300, 2], 150, 528, fp8, gather=33, path=path, epi=epi, pad=2)
    _check_grouped([5, 0, 300, 2], 150, 528, fp8, path=path, epi=epi)


@pytest.mark.parametrize("fp8", [False, True], ids=["int8", "fp8"])
@pytest.mark.parametrize("N,pad", [(7, 1), (129, 7), (250, 6), (257, 7), (1003, 5), (128, 4), (300, 1)])
def test_grouped_output_rows_of_any_stride(N, pad, fp8):
    """16-byte rows whose last columns do not fill 16 bytes, and rows that are not 16-byte."""
    _check_grouped([5, 0, 300, 2], N, 272, fp8, gather=33, path=1, pad=pad)
    _check_grouped([5, 0, 40, 2], N, 272, fp8, path=2, pad=pad, epi="bf16_relu")


@pytest.mark.parametrize("path", [1, 2])
def test_grouped_output_at_an_odd_address(path):
    rng = _rng(15)
    xq, wq = _cuda_of(_codes(rng, (300, 160), False)), _cuda_of(_codes(rng, (2, 96, 160), False))
    xs, ws = torch.rand(300, device="cuda"), torch.rand((2, 96), device="cuda")
    off = _cuda_of(np.array([0, 290, 300], np.int32))
    want = sq.w8a8_gemm_grouped(xq, wq, xs, ws, off, path_hint=path)
    buf = torch.full((300, 104), 9.0, dtype=torch.bfloat16, device="cuda")
    sq.w8a8_gemm_grouped(xq, wq, xs, ws, off, out=buf[:, 1:97], path_hint=path)
    assert torch.equal(buf[:, 1:97], want)
    assert (buf[:, 0] == 9).all() and (buf[:, 97:] == 9).all()


@pytest.mark.parametrize("path", [0, 1, 2])
def test_grouped_rows_before_the_first_group(path):
    _check_grouped([6, 40], 64, 64, path=path, first=9, extra_rows=4)


@pytest.mark.parametrize("path", [1, 2])
def test_grouped_repeats_bit_for_bit(path):
    rng = _rng(12)
    xq, wq = _cuda_of(_codes(rng, (40, 2048), True)), _cuda_of(_codes(rng, (4, 300, 2048), True))
    xs, ws = torch.rand(40, device="cuda"), torch.rand((4, 300), device="cuda")
    off = _cuda_of(np.array([0, 10, 11, 30, 40], np.int32))
    first = sq.fp8_gemm_grouped(xq, wq, xs, ws, off, epi="f32", path_hint=path)
    for _ in range(5):
        assert torch.equal(first, sq.fp8_gemm_grouped(xq, wq, xs, ws, off, epi="f32", path_hint=path))


@pytest.mark.parametrize("path", [1, 2])
def test_grouped_bad_rows_and_offsets(path):
    """Indices outside the tokens give rows of zeros; offsets are clamped to the rows."""
    rng = _rng(13)
    X, N, K, R = 20, 96, 160, 30
    xq, wq = _codes(rng, (X, K), False), _codes(rng, (3, N, K), False)
    row = rng.integers(0, X, R).astype(np.int32)
    bad = [0, 11, 29]
    row[bad] = [-1, X, 2 ** 31 - 1]
    off = np.array([-5, 12, 12, 1000], np.int32)
    out = sq.w8a8_gemm_grouped(_cuda_of(xq), _cuda_of(wq), None, None, _cuda_of(off),
                               row_token=_cuda_of(row), epi="i32", path_hint=path).cpu().numpy()
    a = xq.astype(np.int64)[np.where((row >= 0) & (row < X), row, 0)]
    a[bad] = 0
    assert np.array_equal(out[:12], a[:12] @ wq[0].astype(np.int64).T)
    assert np.array_equal(out[12:], a[12:] @ wq[2].astype(np.int64).T)
    # descending offsets: an empty group, nothing written
    keep = torch.full((R, N), 5, dtype=torch.int32, device="cuda")
    sq.w8a8_gemm_grouped(_cuda_of(xq), _cuda_of(wq), None, None,
                         _cuda_of(np.array([20, 10, 5, 0], np.int32)), row_token=_cuda_of(row),
                         epi="i32", out=keep, path_hint=path)
    assert (keep == 5).all()
    # groups that would overlap: the later one starts where the earlier ended
    out = sq.w8a8_gemm_grouped(_cuda_of(xq), _cuda_of(wq), None, None,
                               _cuda_of(np.array([0, 20, 10, 30], np.int32)), row_token=_cuda_of(row),
                               epi="i32", path_hint=path).cpu().numpy()
    assert np.array_equal(out[:20], a[:20] @ wq[0].astype(np.int64).T)
    assert np.array_equal(out[20:], a[20:] @ wq[2].astype(np.int64).T)


@pytest.mark.parametrize("path", [1, 2])
def test_grouped_running_maximum_crosses_the_warp(path):
    """More experts than a warp has lanes, with offsets that fall back in between."""
    rng = _rng(14)
    E, N, K, R = 70, 40, 64, 200
    off = np.sort(rng.integers(0, R + 1, E + 1)).astype(np.int32)
    off[[10, 33, 40, 64]] = [0, 3, 199, 1]
    run = np.maximum.accumulate(np.clip(off, 0, R))
    xq, wq = _codes(rng, (R, K), False), _codes(rng, (E, N, K), False)
    out = torch.full((R, N), 5, dtype=torch.int32, device="cuda")
    sq.w8a8_gemm_grouped(_cuda_of(xq), _cuda_of(wq), None, None, _cuda_of(off), epi="i32", out=out,
                         path_hint=path)
    want = np.full((R, N), 5, np.int64)
    for e in range(E):
        want[run[e]:run[e + 1]] = xq[run[e]:run[e + 1]].astype(np.int64) @ wq[e].astype(np.int64).T
    assert np.array_equal(out.cpu().numpy(), want)


# ---------------------------------------------------------------------------
# block norm
# ---------------------------------------------------------------------------

NORM = {"none": sq.NORM_NONE, "rms": sq.NORM_RMS, "layer": sq.NORM_LAYER}


def _check_block(M, K, dtype=torch.bfloat16, post="rms", pre="rms", top_k=0, R=None, gate=False,
                 token_gate=False, residual=True, fp8=False, params=True, seed=0, alias=None,
                 pad=0, tweak=None):
    rng = _rng(21, seed, M, K, top_k)
    R = R if R is not None else M * max(1, top_k)
    x = rng.standard_normal((R, K))
    x[:, rng.integers(0, K)] *= 30
    res = rng.standard_normal((M, K)) * 3

    def rows(a):
        t = torch.zeros((a.shape[0], a.shape[1] + pad), dtype=dtype, device="cuda")
        t[:, :a.shape[1]] = _cuda_of(a).to(dtype)
        return t[:, :a.shape[1]]

    xt, rt = rows(x), rows(res) if residual else None
    vec = {}
    for side, kind in (("post", post), ("pre", pre)):
        vec[side + "_gamma"] = rng.uniform(0.5, 1.5, K).astype(np.float32) if params else None
        vec[side + "_beta"] = (rng.standard_normal(K) * 0.1).astype(np.float32) if params and kind == "layer" else None
    g = rng.uniform(-1, 1, K).astype(np.float32) if gate else None
    tg = rng.uniform(0, 1, M).astype(np.float32) if token_gate else None
    tr = w = None
    if top_k:
        tr = rng.integers(0, max(R, 1), (M, top_k)).astype(np.int32)
        w = rng.uniform(0, 1, (M, top_k)).astype(np.float32)
    if tweak:
        tweak(locals())
    x64, r64 = _np64(xt), _np64(rt) if residual else None
    h_out = rt if alias == "residual" else xt if alias == "x" else None
    h, q, s = sq.block_norm_quant_per_token(
        xt, rt, token_row=None if tr is None else _cuda_of(tr), weights=None if w is None else _cuda_of(w),
        post_norm=NORM[post], pre_norm=NORM[pre], gate=None if g is None else _cuda_of(g),
        token_gate=None if tg is None else _cuda_of(tg), residual_scale=0.7, fp8=fp8, h_out=h_out,
        **{k: None if v is None else _cuda_of(v) for k, v in vec.items()})
    if alias:
        assert h is h_out
    hr, dh, y, dy = ref.block_norm(
        x64, r64, tr, w, (post, vec["post_gamma"], vec["post_beta"], 1e-5), g, tg, 0.7,
        (pre, vec["pre_gamma"], vec["pre_beta"], 1e-5))
    hg = _np64(h)
    half = 2.0 ** -9 if dtype == torch.bfloat16 else 2.0 ** -24
    # half a step of the stored type: eps / 2 relative to the value (2^-8 in bf16)
    assert (np.abs(hg - hr) <= dh + 2 * half * (np.abs(hr) + dh)).all()
    vals = ref.E4M3[q.cpu().numpy()] if fp8 else q.cpu().numpy().astype(np.float64)
    ref.check_codes(vals, s.cpu().numpy().astype(np.float64), y, dy, 448.0 if fp8 else 127.0)
    return h, q, s


SHAPES = [(1, 16), (3, 48), (17, 272), (130, 4112), (5, 8192), (4, 9216), (3, 16384), (2, 16400), (2, 32768),
          (1000, 1024)]


@pytest.mark.parametrize("fp8", [False, True], ids=["int8", "fp8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%dx%d" % s)
def test_block_norm_shapes(shape, dtype, fp8):
    _check_block(*shape, dtype=dtype, fp8=fp8, pad=8)
    _check_block(*shape, dtype=dtype, fp8=fp8, top_k=2, post="layer", pre="layer", gate=True)


@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
@pytest.mark.parametrize("top_k", [0, 1, 3, 16])
def test_block_norm_forms(post, pre, top_k):
    for residual, gate, tg, params in ((True, False, False, True), (False, True, True, True),
                                       (True, True, True, False)):
        _check_block(9, 528, post=post, pre=pre, top_k=top_k, residual=residual, gate=gate,
                     token_gate=tg, params=params, fp8=top_k == 3)


def test_block_norm_many_rows():
    _check_block(3000, 2048)
    _check_block(2500, 4096, top_k=2, post="none", token_gate=True)
    _check_block(700, 8192, post="layer", pre="layer", dtype=torch.float32)


@pytest.mark.parametrize("K", [16, 272, 1024, 1040])
@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
@pytest.mark.parametrize("top_k", [0, 1, 4, 5])
def test_block_norm_pipeline_forms(top_k, pre, post, K):
    """Enough rows that every group of the pipeline runs several (five summed rows: without it)."""
    M = 5200 if K < 1024 else 2600

    def tweak(v):
        if top_k:
            v["tr"][::7, 0] = -1
            v["tr"][3] = -1

    for residual, gate, tg, params in ((True, True, False, True), (False, False, True, False)):
        _check_block(M, K, post=post, pre=pre, top_k=top_k, R=700 if top_k else None, gate=gate,
                     token_gate=tg, residual=residual, params=params, fp8=K == 272, tweak=tweak,
                     dtype=torch.float32 if K == 16 else torch.bfloat16, pad=8)


@pytest.mark.parametrize("post", ["none", "rms"])
@pytest.mark.parametrize("residual", [True, False])
def test_block_norm_pipeline_without_codes(post, residual):
    x, res = torch.randn((6000, 512), device="cuda"), torch.randn((6000, 512), device="cuda")
    h, q, s = sq.block_norm_quant_per_token(x, res if residual else None, post_norm=NORM[post], quant=False)
    assert q is None and s is None
    want, *_ = sq.block_norm_quant_per_token(x, res if residual else None, post_norm=NORM[post])
    assert torch.equal(h, want)
    if post == "none":
        assert torch.equal(h, x + res if residual else x)


@pytest.mark.parametrize("alias", ["residual", "x"])
def test_block_norm_in_place_pipelined(alias):
    a = _check_block(5000, 512, alias=alias, pad=16, seed=4)
    b = _check_block(5000, 512, pad=16, seed=4)
    for u, v in zip(a, b):
        assert torch.equal(u, v)


@pytest.mark.parametrize("alias", ["residual", "x"])
def test_block_norm_in_place(alias):
    a = _check_block(400, 1040, alias=alias, pad=16, seed=3)
    b = _check_block(400, 1040, pad=16, seed=3)
    for u, v in zip(a, b):
        assert torch.equal(u, v)


def test_block_norm_missing_rows_are_not_read():
    def tweak(v):
        v["tr"][0] = -1                   # a token none of whose experts took it
        v["tr"][1, 1] = v["R"]            # outside the rows
        v["tr"][2, 0] = -2 ** 31
        v["xt"][5] = float("nan")         # a row no entry names
        v["tr"][v["tr"] == 5] = 6

    _check_block(40, 512, top_k=3, R=60, tweak=tweak)


def test_block_norm_zero_and_tiny_rows():
    def tweak(v):
        v["xt"][0] = 0
        v["rt"][0] = 0
        v["xt"][1] = 1e-30
        v["rt"][1] = 0
        v["xt"][2] = 1e-41
        v["rt"][2] = 0

    for fp8 in (False, True):
        for dtype in (torch.bfloat16, torch.float32):
            _check_block(6, 256, dtype=dtype, pre="rms", post="rms", params=False, fp8=fp8, tweak=tweak)
    h, q, s = sq.block_norm_quant_per_token(torch.zeros((2, 64), device="cuda"), pre_norm=sq.NORM_NONE)
    assert (s == 0).all() and (q == 0).all() and (h == 0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_block_norm_non_finite_rows_show_in_their_scale(bad):
    x = torch.randn((5, 512), device="cuda").to(torch.bfloat16)
    clean = sq.block_norm_quant_per_token(x, pre_norm=sq.NORM_RMS)
    y = x.clone()
    y[2, 100] = bad
    for pre in NORM.values():
        h, q, s = sq.block_norm_quant_per_token(y, pre_norm=pre)
        assert not torch.isfinite(s[2])
        assert torch.isfinite(s[[0, 1, 3, 4]]).all()
    h, q, s = sq.block_norm_quant_per_token(y, pre_norm=sq.NORM_RMS)
    for u, v in zip((h, q, s), clean):
        assert torch.equal(u[[0, 1, 3, 4]], v[[0, 1, 3, 4]])


def test_block_norm_without_codes():
    x = torch.randn((7, 256), device="cuda")
    res = torch.randn((7, 256), device="cuda")
    h, q, s = sq.block_norm_quant_per_token(x, res, residual_scale=2.0, quant=False)
    assert q is None and s is None
    assert torch.equal(h, torch.addcmul(x, res, torch.full_like(res, 2.0)))  # 2 res is exact


# ---------------------------------------------------------------------------
# limits, streams, graphs, the layer
# ---------------------------------------------------------------------------

def test_grouped_equals_the_dense_gemm_of_each_expert():
    rng = _rng(31)
    counts, N, K = [300, 0, 5, 129], 520, 1040
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    xq, wq = _cuda_of(_codes(rng, (off[-1], K), False)), _cuda_of(_codes(rng, (4, N, K), False))
    xs, ws = torch.rand(int(off[-1]), device="cuda"), torch.rand((4, N), device="cuda")
    for epi in ("bf16", "bf16_relu"):
        for path in (1, 2):
            got = sq.w8a8_gemm_grouped(xq, wq, xs, ws, _cuda_of(off), epi=epi, path_hint=path)
            for e in range(4):
                if counts[e]:
                    sl = slice(int(off[e]), int(off[e + 1]))
                    one = sq.w8a8_gemm_dequant(xq[sl].clone(), wq[e], xs[sl].clone(), ws[e].clone(), epi)
                    assert torch.equal(got[sl], one)


@pytest.mark.parametrize("path", [1, 2])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_wait_limit(path, gather):
    """A wait that runs out is an error status, and the next call is right."""
    rng = _rng(32)
    counts, N, K, X = [200, 300], 700, 2048, 500
    off = _cuda_of(np.array([0, 200, 500], np.int32))
    row = _cuda_of(rng.permutation(X).astype(np.int32)) if gather else None
    xq, wq = _cuda_of(_codes(rng, (X, K), False)), _cuda_of(_codes(rng, (2, N, K), False))
    call = lambda: sq.w8a8_gemm_grouped(xq, wq, None, None, off, row_token=row, epi="i32", path_hint=path)  # noqa: E731
    want = call()
    torch.cuda.synchronize()
    assert sq.get_device_error() == 0
    sq.set_wait_limit(1)
    try:
        call()
        assert sq.status_string(sq.get_device_error()).startswith("SQ_ERR_PIPELINE_TIMEOUT")
    finally:
        sq.set_wait_limit(0)
    assert torch.equal(call(), want)
    assert sq.get_device_error() == 0


def test_block_norm_after_a_wait_limit():
    """One probe of a barrier may sleep until its row has landed, so a budget of one may or may
    not run out; either way the call returns, and the next one is right."""
    x = torch.randn((4000, 4096), device="cuda").to(torch.bfloat16)
    res = torch.randn_like(x)
    want = sq.block_norm_quant_per_token(x, res, post_norm=sq.NORM_RMS)
    sq.set_wait_limit(1)
    try:
        sq.block_norm_quant_per_token(x, res, post_norm=sq.NORM_RMS)
        assert sq.get_device_error() in (0, 6)  # SQ_OK, SQ_ERR_PIPELINE_TIMEOUT
    finally:
        sq.set_wait_limit(0)
    for a, b in zip(sq.block_norm_quant_per_token(x, res, post_norm=sq.NORM_RMS), want):
        assert torch.equal(a, b)
    assert sq.get_device_error() == 0


def test_block_norm_pipeline_equals_the_single_row_kernel():
    """The rows of a large batch (pipelined) against the same rows in batches
    too small for the pipeline: the same values, sums in another order."""
    x = torch.randn((8000, 1040), device="cuda")
    res = torch.randn_like(x)
    rows = torch.randint(-1, 8000, (5000, 3), device="cuda", dtype=torch.int32)
    w = torch.rand((5000, 3), device="cuda")
    g = torch.rand(1040, device="cuda")
    kw = dict(post_norm=sq.NORM_LAYER, post_gamma=g, gate=g, pre_gamma=g)
    h, q, s = sq.block_norm_quant_per_token(x, res[:5000], token_row=rows, weights=w, **kw)
    h1, q1, s1 = sq.block_norm_quant_per_token(x, res[:100], token_row=rows[:100].contiguous(),
                                               weights=w[:100].contiguous(), **kw)
    # both within 300 roundings of the same number (|h| of order 1)
    assert (h[:100] - h1).abs().max() <= 300 * 2.0 ** -24 * max(1.0, float(h1.abs().max()))
    assert (q[:100].int() - q1.int()).abs().max() <= 1


def _layer(fmt, T=70, E=8, H=256, I=160, top_k=2, seed=0, **kw):
    from w8a8_int8_quantized_norm_b200 import moe

    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    gu, dn = (rand(E, 2 * I, H) * 0.05).to(torch.bfloat16), (rand(E, H, I) * 0.05).to(torch.bfloat16)
    x, res = rand(T, H).to(torch.bfloat16), rand(T, H).to(torch.bfloat16)
    x[:, 3] *= 40
    gamma = torch.rand(H, device="cuda", generator=gen) + 0.5
    layer = moe.MoELayer(gu, dn, top_k, fmt=fmt, **kw)
    act = sq.calibrate_absmax(x, sq.NORM_RMS, gamma)
    layer.prepare(act, 0.5, gamma)
    norm = sq.norm_smooth_quant_per_token if fmt == "int8" else sq.norm_smooth_quant_per_token_fp8
    logits = rand(T, E)
    Xq, xs = norm(x, sq.NORM_RMS, layer.gamma)
    block = dict(post_norm=sq.NORM_RMS, post_gamma=gamma, pre_norm=sq.NORM_RMS, pre_gamma=gamma,
                 residual_scale=0.5)
    return layer, x, gamma, Xq, xs, logits, res, block


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_layer_stage_by_stage(fmt):
    import oracle

    layer, x, gamma, Xq, xs, logits, res, block = _layer(fmt)
    logits[60:] = -float("inf")  # a padded tail
    h, q, s = layer.forward(Xq, xs, logits, res, **block)
    st = layer.stages
    w, e, off, row, tok, bound = ref.route(_np64(logits), 2)
    r = st["route"]
    for got, want in ((r.experts, e), (r.offsets, off), (r.row_token, row), (r.token_row, tok)):
        assert np.array_equal(got.cpu().numpy(), want)
    n = int(off[-1])
    fp8 = fmt == "fp8"
    a = _values(Xq.cpu().numpy(), fp8) * _np64(xs)[:, None]
    wide = _values(layer.gate_up_q.cpu().numpy(), fp8) * _np64(layer.gate_up_scale)[:, :, None]
    narrow = _values(layer.down_q.cpu().numpy(), fp8) * _np64(layer.down_scale)[:, :, None]
    ha = _values(st["Hq"].cpu().numpy(), fp8) * _np64(st["h_scale"])[:, None]
    gu, y = _np64(st["gate_up"]), _np64(st["down"])
    for ex in range(8):
        sl = slice(off[ex], off[ex + 1])
        for got, left, right in ((gu[sl], a[row[sl]], wide[ex]), (y[sl], ha[sl], narrow[ex])):
            want = left @ right.T
            # accumulation (FP8) and the two scales' roundings, then bf16's half step
            slack = (31 + 8 + 4) * 2.0 ** -23 * (np.abs(left) @ np.abs(right).T)
            assert (np.abs(got - want) <= slack + 2.0 ** -8 * (np.abs(want) + slack)).all()
    if not fp8:
        bits = st["gate_up"][:n].view(torch.int16).cpu().numpy().view(np.uint16)
        hq, hs, _ = oracle.silu_mul_quant(bits)
        assert np.array_equal(st["Hq"][:n].cpu().numpy(), hq)
        assert np.array_equal(st["h_scale"][:n].cpu().numpy(), hs)
    g = gamma.cpu().numpy()
    hr, dh, yr, dy = ref.block_norm(y, _np64(res), tok, r.weights.cpu().numpy().astype(np.float64),
                                    ("rms", g, None, 1e-5), None, None, 0.5, ("rms", g, None, 1e-5))
    assert (np.abs(_np64(h) - hr) <= dh + 2.0 ** -8 * (np.abs(hr) + dh)).all()
    vals = _values(q.cpu().numpy(), fp8)
    ref.check_codes(vals, _np64(s), yr, dy, 448.0 if fp8 else 127.0)


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_layer_is_near_the_unquantised_experts(fmt):
    """The whole layer against fp64 experts on the bf16 weights: smoothed 8-bit codes keep the
    sum of the experts within a few percent (a wrong fold, expert or weight is far outside)."""
    layer, x, gamma, Xq, xs, logits, res, _ = _layer(fmt, T=64)
    h, _, _ = layer.forward(Xq, xs, logits, None, post_norm=sq.NORM_NONE, quant=False)
    X = _np64(x)
    n = X / np.sqrt((X * X).mean(1, keepdims=True) + 1e-5) * gamma.cpu().numpy()
    w, e, *_ = ref.route(_np64(logits), 2)
    gu, dn = _np64(layer.gate_up), _np64(layer.down)
    want = np.zeros_like(X)
    for t in range(64):
        for j in range(2):
            z = gu[e[t, j]] @ n[t]
            g, u = z[:160], z[160:]
            want[t] += w[t, j] * (dn[e[t, j]] @ (g / (1 + np.exp(-g)) * u))
    rel = np.linalg.norm(_np64(h) - want) / np.linalg.norm(want)
    # int8: four roundings of about step / sqrt(12), step = max / 127; e4m3: 2^-4 / sqrt(3) each
    assert rel < (0.05 if fmt == "int8" else 0.12)


def test_layer_without_tokens():
    layer, x, gamma, Xq, xs, logits, res, block = _layer("int8", T=4)
    h, q, s = layer.forward(Xq[:0], xs[:0], logits[:0], res[:0], **block)
    assert h.shape == (0, 256) and q.shape == (0, 256) and s.shape == (0,)


def test_layer_with_every_token_masked():
    layer, x, gamma, Xq, xs, logits, res, block = _layer("int8", T=40)
    logits.fill_(-float("inf"))
    h, q, s = layer.forward(Xq, xs, logits, res, **dict(block, post_norm=sq.NORM_NONE, post_gamma=None))
    assert torch.equal(h, (res.float() * 0.5).to(torch.bfloat16))


def test_layer_in_a_graph_and_on_another_stream():
    layer, x, gamma, Xq, xs, logits, res, block = _layer("int8", T=33)
    want = [t.clone() for t in layer.forward(Xq, xs, logits, res, **block)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = layer.forward(Xq, xs, logits, res, stream=side, **block)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # two captured graphs, replayed in turn on changed inputs
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = layer.forward(Xq, xs, logits, res, **block)
        graphs.append((g, out))
    logits.copy_(logits.flip(0))
    fresh = [t.clone() for t in layer.forward(Xq, xs, logits, res, **block)]
    for g, out in graphs + graphs[:1]:
        for t in out:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, fresh):
            assert torch.equal(a, b)


def test_calls_on_two_streams_at_once():
    """No call shares scratch with another: two streams at once give what each gives alone."""
    logits = [torch.randn((5000, 64), device="cuda") for _ in range(2)]
    x = [torch.randn((4000, 2048), device="cuda").to(torch.bfloat16) for _ in range(2)]
    alone = [(sq.moe_route(l, 6), sq.block_norm_quant_per_token(v, v)) for l, v in zip(logits, x)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            got[i].append((sq.moe_route(logits[i], 6, stream=st),
                           sq.block_norm_quant_per_token(x[i], x[i], stream=st)))
    torch.cuda.synchronize()
    for i in range(2):
        for r, b in got[i]:
            for u, v in zip(tuple(r) + tuple(b), tuple(alone[i][0]) + tuple(alone[i][1])):
                assert torch.equal(u, v)


def test_binding_refusals():
    x = torch.randn((4, 64), device="cuda")
    with pytest.raises(ValueError):
        sq.moe_route(x, 65)
    with pytest.raises(ValueError):
        sq.moe_route(x, 2, score="relu")
    with pytest.raises(ValueError):
        sq.moe_route(x, 2, score="sigmoid", bias=torch.zeros(63, device="cuda"))
    with pytest.raises(sq.SQError):
        sq.moe_route(x, 2, bias=torch.zeros(64, device="cuda"))  # softmax takes none
    with pytest.raises(sq.SQError):
        sq.moe_route(torch.randn((100, 64), device="cuda"), 2,
                     workspace=torch.empty(4, dtype=torch.uint8, device="cuda"))
    codes, w = torch.zeros((4, 64), dtype=torch.int8, device="cuda"), \
        torch.zeros((2, 8, 64), dtype=torch.int8, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    ok = (torch.zeros(4, device="cuda"), torch.zeros((2, 8), device="cuda"))
    with pytest.raises(ValueError):
        sq.w8a8_gemm_grouped(codes, w, *ok, off.long())
    with pytest.raises(ValueError):
        sq.w8a8_gemm_grouped(codes, w, *ok, off[:2])
    with pytest.raises(ValueError):
        sq.w8a8_gemm_grouped(codes, w, *ok, off, out=torch.zeros((4, 9), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        sq.w8a8_gemm_grouped(codes.view(torch.uint8), w, *ok, off)
    with pytest.raises(sq.SQError):
        sq.w8a8_gemm_grouped(codes, w, None, None, off)  # bf16 needs scales
    with pytest.raises(ValueError):
        sq.block_norm_quant_per_token(x, token_row=torch.zeros((4, 2), dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        sq.block_norm_quant_per_token(x, x.double())
    with pytest.raises(sq.SQError):
        sq.block_norm_quant_per_token(x, h_out=x, token_row=torch.zeros((4, 1), dtype=torch.int32, device="cuda"),
                                      weights=torch.zeros((4, 1), device="cuda"))
    with pytest.raises(sq.SQError):
        sq.block_norm_quant_per_token(torch.zeros((4, 72), device="cuda"))  # K % 16


# ---------------------------------------------------------------------------
# addresses past 32 bits
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("path", [1, 2])
def test_grouped_output_past_32_bits(path):
    """R N > 2^31 outputs: the last rows are right, and so are the first."""
    R, N, K = 70000, 32768, 16
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    x = torch.randint(-127, 128, (R, K), generator=gen, device="cuda", dtype=torch.int8)
    w = torch.randint(-127, 128, (2, N, K), generator=gen, device="cuda", dtype=torch.int8)
    off = _cuda_of(np.array([0, 100, R], np.int32))
    one = torch.ones(R, device="cuda")
    out = sq.w8a8_gemm_grouped(x, w, one, torch.ones((2, N), device="cuda"), off, path_hint=path)
    for rows, e in ((slice(0, 50), 0), (slice(R // 2, R // 2 + 50), 1), (slice(R - 50, R), 1)):
        want = (x[rows].double() @ w[e].double().T).float().to(torch.bfloat16)
        assert torch.equal(out[rows], want)


@pytest.mark.parametrize("path", [1, 2])
def test_grouped_weights_past_32_bits(path):
    E, N, K = 70, 8192, 4096
    gen = torch.Generator(device="cuda")
    gen.manual_seed(6)
    w = torch.randint(-127, 128, (E, N, K), generator=gen, device="cuda", dtype=torch.int8)
    x = torch.randint(-127, 128, (40, K), generator=gen, device="cuda", dtype=torch.int8)
    off = np.zeros(E + 1, np.int32)
    off[36:] = 10
    off[E:] = 40  # rows for experts 35 and 69
    out = sq.w8a8_gemm_grouped(x, w, None, None, _cuda_of(off), epi="i32", path_hint=path)
    for rows, e in ((slice(0, 10), 35), (slice(10, 40), 69)):
        assert torch.equal(out[rows].double(), x[rows].double() @ w[e].double().T)


@pytest.mark.parametrize("top_k", [0, 2])
def test_block_norm_past_32_bits(top_k):
    """M K > 2^31 values: sampled rows equal the same rows in a batch of their own
    (as far as the sums' order allows)."""
    M, K = 264000, 8192
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7)
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    pick = torch.tensor([0, 1, M // 2, M - 2, M - 1], device="cuda")
    rows = w = None
    if top_k:
        rows = torch.randint(0, M, (M, 2), device="cuda", dtype=torch.int32, generator=gen)
        w = torch.rand((M, 2), device="cuda", generator=gen)
    h, q, s = sq.block_norm_quant_per_token(x, x, token_row=rows, weights=w, post_norm=sq.NORM_RMS)
    x64, r64 = _np64(x[pick]), _np64(x[pick])
    if top_k:
        x64 = sum(_np64(x[rows[pick][:, j].long()]) * _np64(w[pick])[:, j:j + 1] for j in range(2))
    hr, dh, y, dy = ref.block_norm(x64, r64, None, None, ("rms", None, None, 1e-5), None, None, 1.0,
                                   ("rms", None, None, 1e-5))
    dh, dy = dh * 1.1 + 4 * ref.U * np.abs(hr).max(), dy * 1.1 + 8 * ref.U * np.abs(y).max()  # the sum of two rows
    assert (np.abs(_np64(h[pick]) - hr) <= dh + 2.0 ** -8 * (np.abs(hr) + dh)).all()
    ref.check_codes(_np64(q[pick].float()), _np64(s[pick]), y, dy, 127.0)
