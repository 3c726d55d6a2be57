"""The operators of a layer of experts at their edges: waits that run out, memory of the right
stream, values near the ends of fp32, layouts inside one buffer."""
import copy

import numpy as np
import pytest
import torch

from w8a8_int8_quantized_norm_b200 import sq

import _moe_reference as ref

pytestmark = pytest.mark.gpu

TIMEOUT = 6  # SQ_ERR_PIPELINE_TIMEOUT


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    sq.lib()
    assert sq.get_device_error() == 0
    yield
    sq.set_wait_limit(0)
    assert sq.get_device_error() == 0


def _rng(*key):
    return np.random.default_rng([17, *key])


def _cuda_of(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def _np64(t):
    return t.double().cpu().numpy()


# ---------------------------------------------------------------------------
# block norm: waits that run out
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("limit", [1, 2, 4])
@pytest.mark.parametrize("quant", [True, False])
@pytest.mark.parametrize("pre", [sq.NORM_NONE, sq.NORM_RMS])
@pytest.mark.parametrize("top_k", [0, 2])
def test_block_norm_wait_limit(top_k, pre, quant, limit):
    """A wait that runs out is an error status: its group starts no further copy and leaves, and
    the next call is right.  A limit of 1 allows no probe and always runs out; 2 and 4 allow one
    and three that do not sleep, so that groups give up at some later row, or not at all."""
    M, K = 6000, 2048  # ten rows or more for every group
    x = torch.randn((M * max(1, top_k), K), device="cuda").to(torch.bfloat16)
    res = torch.randn((M, K), device="cuda").to(torch.bfloat16)
    kw = dict(post_norm=sq.NORM_RMS, pre_norm=pre, quant=quant)
    if top_k:
        kw.update(token_row=torch.randperm(M * top_k, device="cuda").to(torch.int32).view(M, top_k),
                  weights=torch.rand((M, top_k), device="cuda"))
    want = sq.block_norm_quant_per_token(x, res, **kw)
    torch.cuda.synchronize()
    assert sq.get_device_error() == 0
    sq.set_wait_limit(limit)
    try:
        sq.block_norm_quant_per_token(x, res, **kw)
        status = sq.get_device_error()
    finally:
        sq.set_wait_limit(0)
    assert status == TIMEOUT if limit == 1 else status in (0, TIMEOUT)
    got = sq.block_norm_quant_per_token(x, res, **kw)
    assert sq.get_device_error() == 0
    for a, b in zip(got, want):
        assert (a is None and b is None) or torch.equal(a, b)


# ---------------------------------------------------------------------------
# memory of the stream that the work runs on
# ---------------------------------------------------------------------------

class _Allocations:
    """Records the current stream of every torch.empty / torch.zeros on the GPU."""

    def __init__(self, monkeypatch):
        self.streams = []
        for name in ("empty", "zeros"):
            monkeypatch.setattr(torch, name, self._recording(getattr(torch, name)))

    def _recording(self, make):
        def call(*args, **kw):
            self.streams.append(torch.cuda.current_stream())
            return make(*args, **kw)
        return call


def _binding_calls():
    """Every call of the binding that allocates, as a function of the stream alone."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    M, N, K = 40, 96, 256
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, W = rand(M, K).to(torch.bfloat16), rand(N, K).to(torch.bfloat16)
    gu = rand(M, 2 * K).to(torch.bfloat16)
    vec, amax = rand(K).abs() + 0.5, rand(M).abs() + 5
    xq = torch.randint(-127, 128, (M, K), generator=gen, device="cuda", dtype=torch.int8)
    wq = torch.randint(-127, 128, (N, K), generator=gen, device="cuda", dtype=torch.int8)
    x8, w8 = xq.view(torch.uint8) & 0x77, wq.view(torch.uint8) & 0x77
    xs, ws = rand(M).abs(), rand(N).abs()
    acc = torch.randint(-1000, 1000, (M, N), generator=gen, device="cuda", dtype=torch.int32)
    idx = torch.arange(K, device="cuda", dtype=torch.int32)
    count = torch.full((1,), 3, device="cuda", dtype=torch.int32)
    one = vec.abs().max().reshape(1)
    logits = rand(M, 8)
    off = _cuda_of(np.array([0, 10, M], np.int32))
    we, wse = wq.view(2, N // 2, K), ws.view(2, N // 2)
    rms = sq.NORM_RMS
    # long in K, so that the decode GEMM splits and takes a workspace
    xl, wl = xq.repeat(1, 64)[:16].contiguous(), wq.repeat(1, 64)
    return {
        "calibrate_absmax": lambda s: sq.calibrate_absmax(x, rms, vec, stream=s),
        "compute_smooth_scales": lambda s: sq.compute_smooth_scales(vec, [W], 0.5, gamma=vec, beta=vec, stream=s),
        "weight_column_max": lambda s: sq.weight_column_max([W], stream=s),
        "smooth_scales_from_maxima": lambda s: sq.smooth_scales_from_maxima(vec, vec, 0.5, gamma=vec, beta=vec,
                                                                            stream=s),
        "smooth_quantize_weights": lambda s: sq.smooth_quantize_weights(W, vec, stream=s),
        "smooth_quantize_weights_fp8": lambda s: sq.smooth_quantize_weights_fp8(W, vec, stream=s),
        "smooth_quantize_weights_per_tensor": lambda s: sq.smooth_quantize_weights_per_tensor(W, vec, stream=s),
        "norm_smooth_quant_per_token": lambda s: sq.norm_smooth_quant_per_token(x, rms, vec, stream=s),
        "norm_smooth_quant_per_token_fp8": lambda s: sq.norm_smooth_quant_per_token_fp8(x, rms, vec, stream=s),
        "norm_smooth_absmax": lambda s: sq.norm_smooth_absmax(x, rms, vec, stream=s),
        "norm_smooth_quant_per_tensor": lambda s: sq.norm_smooth_quant_per_tensor(x, rms, one, vec, stream=s),
        "quant_per_token_given_absmax": lambda s: sq.quant_per_token_given_absmax(x, amax, stream=s),
        "row_absmax": lambda s: sq.row_absmax(x, stream=s),
        "dequant_i32": lambda s: sq.dequant_i32(acc, xs, ws, stream=s),
        "llmint8_outliers": lambda s: sq.llmint8_outliers(vec, 1.0, stream=s)[::2],
        "llmint8_combine": lambda s: sq.llmint8_combine(acc, xs, ws, x, W, idx, count, stream=s),
        "silu_mul_quant_per_token": lambda s: sq.silu_mul_quant_per_token(gu, stream=s),
        "silu_mul_quant_per_token_fp8": lambda s: sq.silu_mul_quant_per_token(gu, stream=s, fp8=True),
        "fp8_gemm_dequant": lambda s: sq.fp8_gemm_dequant(x8, w8, xs, ws, stream=s),
        "w8a8_gemm_dequant": lambda s: sq.w8a8_gemm_dequant(xq, wq, xs, ws, stream=s),
        "w8a8_gemm_dequant_split": lambda s: sq.w8a8_gemm_dequant(xl, wl, None, None, "i32", path_hint=2,
                                                                  split_k=4, stream=s),
        "w8a8_gemm_dequant_rowmax": lambda s: sq.w8a8_gemm_dequant_rowmax(xq, wq, xs, ws, path_hint=1, stream=s),
        "linear_w8a8": lambda s: sq.linear_w8a8(x, rms, vec, None, 1e-5, wq, ws, stream=s),
        "moe_route": lambda s: sq.moe_route(logits, 2, stream=s),
        "w8a8_gemm_grouped": lambda s: sq.w8a8_gemm_grouped(xq, we, xs, wse, off, stream=s),
        "fp8_gemm_grouped": lambda s: sq.fp8_gemm_grouped(x8, w8.view(2, N // 2, K), xs, wse, off, stream=s),
        "block_norm_quant_per_token": lambda s: sq.block_norm_quant_per_token(x, x, stream=s),
    }


def _tensors(got):
    return [got] if torch.is_tensor(got) else [t for t in got if t is not None]


CALLS = ["calibrate_absmax", "compute_smooth_scales", "weight_column_max", "smooth_scales_from_maxima",
         "smooth_quantize_weights", "smooth_quantize_weights_fp8", "smooth_quantize_weights_per_tensor",
         "norm_smooth_quant_per_token", "norm_smooth_quant_per_token_fp8", "norm_smooth_absmax",
         "norm_smooth_quant_per_tensor", "quant_per_token_given_absmax", "row_absmax", "dequant_i32",
         "llmint8_outliers", "llmint8_combine", "silu_mul_quant_per_token", "silu_mul_quant_per_token_fp8",
         "fp8_gemm_dequant", "w8a8_gemm_dequant", "w8a8_gemm_dequant_split", "w8a8_gemm_dequant_rowmax",
         "linear_w8a8", "moe_route", "w8a8_gemm_grouped", "fp8_gemm_grouped", "block_norm_quant_per_token"]


@pytest.mark.parametrize("name", CALLS)
def test_outputs_and_scratch_come_from_the_stream_of_the_call(name, monkeypatch):
    """A block of the caller's stream's memory may still be in use there, and nothing orders that
    stream against the call's: what a call allocates is the memory of the stream it runs on."""
    call = _binding_calls()[name]
    want = [t.clone() for t in _tensors(call(None))]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    seen = _Allocations(monkeypatch)
    got = _tensors(call(side))
    side.synchronize()
    assert seen.streams and all(s == side for s in seen.streams)
    assert torch.cuda.current_stream() != side
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def _layer(fmt, T=70, E=8, H=256, I=160, top_k=2, **kw):
    from w8a8_int8_quantized_norm_b200 import moe

    gen = torch.Generator(device="cuda")
    gen.manual_seed(11)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    gu, dn = (rand(E, 2 * I, H) * 0.05).to(torch.bfloat16), (rand(E, H, I) * 0.05).to(torch.bfloat16)
    x, res, gamma = rand(T, H).to(torch.bfloat16), rand(T, H).to(torch.bfloat16), rand(H).abs() + 0.5
    layer = moe.MoELayer(gu, dn, top_k, fmt=fmt, **kw)
    act = sq.calibrate_absmax(x, sq.NORM_RMS, gamma)
    layer.prepare(act, 0.5, gamma)
    norm = sq.norm_smooth_quant_per_token if fmt == "int8" else sq.norm_smooth_quant_per_token_fp8
    Xq, xs = norm(x, sq.NORM_RMS, layer.gamma)
    return layer, act, gamma, Xq, xs, rand(T, E), res


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_layer_memory_comes_from_the_stream_of_the_call(fmt, monkeypatch):
    layer, act, gamma, Xq, xs, logits, res = _layer(fmt)
    want = [t.clone() for t in layer.forward(Xq, xs, logits, res)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    seen = _Allocations(monkeypatch)
    layer.prepare(act, 0.5, gamma, stream=side)
    got = layer.forward(Xq, xs, logits, res, stream=side)
    side.synchronize()
    assert len(seen.streams) > 10 and all(s == side for s in seen.streams)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_layer_passes_in_a_row_beside_the_caller_stream(fmt):
    """Passes on a side stream without a wait between them, while the caller's stream allocates,
    overwrites and frees blocks of the stages' sizes."""
    layer, act, gamma, Xq, xs, logits, res = _layer(fmt, T=2000, H=512, I=512)
    want = [t.clone() for t in layer.forward(Xq, xs, logits, res)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = []
    for _ in range(20):
        outs.append(layer.forward(Xq, xs, logits, res, stream=side))
        for n in (2000 * 2 * 1024 * 2, 2000 * 2 * 512, 2000 * 2 * 4):
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
    torch.cuda.synchronize()
    for got in outs:
        for a, b in zip(got, want):
            assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# the layer: what a pass leaves behind
# ---------------------------------------------------------------------------

def test_layers_hold_no_stages_of_earlier_passes():
    """A model of many layers, each pass fed by the one before: the stages of a pass go with its h,
    so that memory does not grow with the layers."""
    T, H, I, k = 1000, 256, 512, 2
    layer, act, gamma, Xq, xs, logits, res = _layer("int8", T=T, H=H, I=I, top_k=k)
    layers = [layer] + [_layer("int8", T=T, H=H, I=I, top_k=k)[0] for _ in range(7)]
    one = T * k * (2 * I * 2 + I + H * 2)  # bytes of a pass's gate/up rows, codes and down rows
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    h, q, s = res, Xq, xs
    for l in layers:
        h, q, s = l.forward(q, s, logits, h)
    assert torch.cuda.memory_allocated() - before < 2 * one
    assert all(l.stages is None for l in layers[:-1])
    assert layers[-1].stages is h.stages
    assert set(h.stages) == {"route", "gate_up", "Hq", "h_scale", "down"}
    assert copy.deepcopy(layers[-1]).stages is None
    del h
    assert layers[-1].stages is None


def test_layer_without_stages_leaves_its_results_alone():
    layer, act, gamma, Xq, xs, logits, res = _layer("fp8", keep_stages=False)
    want = _layer("fp8")[0].forward(Xq, xs, logits, res)
    layer.forward(Xq, xs, logits, res)
    before = torch.cuda.memory_allocated()
    got = layer.forward(Xq, xs, logits, res)
    left = torch.cuda.memory_allocated() - before
    assert left <= sum(-(-t.numel() * t.element_size() // 512) * 512 for t in got)
    assert layer.stages is None and not hasattr(got[0], "stages")
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_two_threads_on_one_layer_keep_their_own_stages():
    import threading

    layer, act, gamma, Xq, xs, logits, res = _layer("int8")
    torch.cuda.synchronize()
    ins = [logits, logits.flip(0).contiguous()]
    got = [None, None]

    def run(i):
        stream = torch.cuda.Stream()
        for _ in range(10):
            got[i] = layer.forward(Xq, xs, ins[i], res, stream=stream)
        stream.synchronize()

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(2):
        want = layer.forward(Xq, xs, ins[i], res)
        for a, b in zip(got[i], want):
            assert torch.equal(a, b)
        mine, its = got[i][0].stages, want[0].stages
        assert torch.equal(mine["route"].experts, its["route"].experts)
        n = int(its["route"].offsets[-1])
        assert torch.equal(mine["down"][:n], its["down"][:n])


# ---------------------------------------------------------------------------
# matrices without rows
# ---------------------------------------------------------------------------

def test_a_matrix_without_rows_has_no_stride():
    """numpy's empty arrays have strides of 0: no rows, so nothing is refused and nothing written.
    With rows the columns still have to follow one another."""
    x = torch.from_numpy(np.empty((0, 64), np.float32)).cuda()
    odd = torch.empty_strided((0, 64), (1, 7), dtype=torch.float32, device="cuda")
    for t in (x, odd):
        q, s = sq.norm_smooth_quant_per_token(t, sq.NORM_RMS)
        assert q.shape == (0, 64) and s.shape == (0,)
        assert sq.row_absmax(t).shape == (0,)
        q, s = sq.silu_mul_quant_per_token(t.to(torch.bfloat16))
        assert q.shape == (0, 32) and s.shape == (0,)
        h, q, s = sq.block_norm_quant_per_token(t)
        assert h.shape == q.shape == (0, 64) and s.shape == (0,)
        assert (sq.moe_route(t, 2).offsets == 0).all()
    strided = torch.zeros((4, 128), device="cuda")[:, ::2]
    for call in (lambda: sq.norm_smooth_quant_per_token(strided, sq.NORM_RMS), lambda: sq.row_absmax(strided),
                 lambda: sq.block_norm_quant_per_token(strided), lambda: sq.moe_route(strided, 2)):
        with pytest.raises(ValueError, match="unit column stride"):
            call()


# ---------------------------------------------------------------------------
# router: scores below fp32's range
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("use_bias", [False, True])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_sigmoid_of_far_negative_logits(renorm, use_bias):
    """Below about -88 exp(-l) overflows fp32, below -104 the score underflows; the ratios of the
    chosen scores are ordinary numbers down to where 64 bits end (-708)."""
    rng = _rng(1)
    E, k = 40, 6
    l = rng.standard_normal((12, E))
    l[0] = rng.uniform(-100, -87, E)
    l[1] = rng.uniform(-300, -90, E)
    l[2] = rng.uniform(-700, -600, E)
    l[3, :36] = -95 + rng.standard_normal(36)  # four of N(0, 1) first
    l[4] = -88.5
    l[5] = -200 - np.arange(E)
    l[5, 7] = -5
    l[6] = -1000
    l[7] = np.finfo(np.float32).min
    l[8] = rng.uniform(-140, -120, E)
    l[8, 3:] = -np.inf                         # three left
    l[9] = rng.uniform(-60, -1e-3, E)
    l[10] = rng.uniform(60, 100, E)
    bias = rng.standard_normal(E).astype(np.float32) if use_bias else None
    logits = l.astype(np.float32)
    r = sq.moe_route(_cuda_of(logits), k, score="sigmoid", bias=None if bias is None else _cuda_of(bias),
                     renormalize=renorm, scale=2.5)
    w, e, *_, bound = ref.route(logits.astype(np.float64), k, "sigmoid", bias, renorm, 2.5)
    assert np.array_equal(r.experts.cpu().numpy(), e)
    g = _np64(r.weights)
    # a chosen score relative to the largest: exp 4 U, its argument's rounding taken back with
    # 2 U, 1 + exp(l) 5 U, quotient 1 U; the sum 5 U, the division and the scale 2 U: 19 U, below
    # the reference's bound (12 + E) U.  Below the normal range: a multiple of 2^-149.
    assert (np.abs(g - w) <= bound * np.abs(w) + 2.0 ** -126).all()
    if renorm:
        assert np.allclose(g[[0, 1, 2, 4, 8]].sum(1), 2.5, rtol=1e-5)
        assert (g[[6, 7]] == 0).all()  # scores of 0


# ---------------------------------------------------------------------------
# block norm: rows whose squares leave fp32
# ---------------------------------------------------------------------------

def _extreme_rows(M, K, dtype, layer):
    """Rows of finite values at both ends of fp32, the first ones each of another kind, in the
    stored values of dtype."""
    rng = _rng(2, K)
    x = rng.standard_normal((M, K))
    x[0] *= 1e25
    x[1] *= 1e35
    x[2] *= 3e-30
    x[3] = 0
    x[3, 5] = 3e38                    # one value near the largest, a row of zeros
    x[4] = 1e19
    x[4, ::2] = -1e19                 # squares just in range, their sum not
    x[5] = rng.uniform(1, 2, K) * 1e36  # the plain sum leaves fp32 too (LayerNorm's mean)
    x[6] *= 1e-38
    x[7, :K // 2] *= 1e21             # the sum of the squares would hide the other half
    return _cuda_of(x).to(dtype)


@pytest.mark.parametrize("fp8", [False, True], ids=["int8", "fp8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("M,K", [(9, 512), (5, 8192), (9, 9216), (3, 32768), (4000, 512), (2500, 4096)])
def test_block_norm_of_rows_whose_squares_leave_fp32(M, K, kind, dtype, fp8):
    """Statistics of finite rows never overflow or vanish: the row's norm, codes and scale are those
    of the definition, as sq.norm_smooth_quant_per_token's are."""
    norm = {"rms": sq.NORM_RMS, "layer": sq.NORM_LAYER}[kind]
    rows = min(M, 8)
    x = _extreme_rows(max(M, 8), K, dtype, kind == "layer")[:M].contiguous()
    keep = np.r_[0:rows, max(rows, M - 4):M]
    for eps in (1e-5, 0.0):
        for post, pre in ((True, False), (False, True), (True, True)):
            h, q, s = sq.block_norm_quant_per_token(
                x, None, post_norm=norm if post else sq.NORM_NONE, post_eps=eps,
                pre_norm=norm if pre else sq.NORM_NONE, pre_eps=eps, fp8=fp8)
            name = lambda on: (kind if on else "none", None, None, eps)  # noqa: E731
            with np.errstate(all="ignore"):
                hr, dh, y, dy = ref.block_norm(_np64(x[keep]), post=name(post), pre=name(pre))
            half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -23
            # (below the normal range h is rounded to a multiple of the type's smallest number)
            tiny = 2.0 ** -133 if dtype == torch.bfloat16 else 2.0 ** -149
            assert (np.abs(_np64(h[keep]) - hr) <= dh + half * (np.abs(hr) + dh) + tiny).all()
            vals = ref.E4M3[q[keep].cpu().numpy()] if fp8 else q[keep].cpu().numpy().astype(np.float64)
            ref.check_codes(vals, _np64(s[keep]), y, dy + 2.0 ** -149, 448.0 if fp8 else 127.0)


def test_block_norm_of_extreme_rows_equals_the_norm_call():
    """Without a norm behind the block the call is sq.norm_smooth_quant_per_token's, whose sums
    are fp64: the same scales but for fp32 roundings, on both kernels."""
    for M, K in ((12, 1040), (4000, 512)):
        x = _extreme_rows(M, K, torch.float32, False)
        _, q, s = sq.block_norm_quant_per_token(x, pre_norm=sq.NORM_RMS)
        q1, s1 = sq.norm_smooth_quant_per_token(x, sq.NORM_RMS)
        assert torch.isfinite(s).all() and (s > 0).all()
        assert ((s - s1).abs() <= 100 * 2.0 ** -24 * s1).all()
        assert (q.int() - q1.int()).abs().max() <= 1


# ---------------------------------------------------------------------------
# errors of earlier calls
# ---------------------------------------------------------------------------

AFTER_AN_ERROR = """
import torch
from w8a8_int8_quantized_norm_b200 import sq

xq = torch.randint(-127, 128, (600, 128), device="cuda", dtype=torch.int8)
wq = torch.randint(-127, 128, (2, 256, 128), device="cuda", dtype=torch.int8)
off = torch.tensor([0, 250, 600], device="cuda", dtype=torch.int32)
torch.cuda.synchronize()
try:  # a synchronisation inside a capture is an error of the host's call, and ends the capture
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        status = sq.get_device_error()
except RuntimeError:
    pass
assert sq.status_string(status).startswith("SQ_ERR_CUDA"), status
for path in (1, 2):
    out = sq.w8a8_gemm_grouped(xq, wq, None, None, off, epi="i32", path_hint=path)
    for e, rows in ((0, slice(0, 250)), (1, slice(250, 600))):
        assert torch.equal(out[rows].double(), xq[rows].double() @ wq[e].double().T)
out = sq.w8a8_gemm_dequant(xq, wq[0], None, None, "i32", path_hint=1)
assert torch.equal(out.double(), xq.double() @ wq[0].double().T)
print("right after the error")
"""


def test_grouped_does_not_report_an_earlier_error():
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", AFTER_AN_ERROR], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "right after the error" in r.stdout, r.stdout + r.stderr[-2000:]


# ---------------------------------------------------------------------------
# block norm: rows side by side in one buffer
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("M", [7, 5000])
@pytest.mark.parametrize("order", [(0, 1, 2), (2, 0, 1), (1, 2, 0)])
def test_block_norm_on_columns_of_one_buffer(order, M):
    """x, residual and h_out as column ranges of one buffer share no byte, and a gap between them
    stays as it was."""
    K, gap = 528, 16
    buf = torch.randn((M, 3 * (K + gap)), device="cuda").to(torch.bfloat16)
    x, res, h = (buf[:, i * (K + gap):i * (K + gap) + K] for i in order)
    kw = dict(post_norm=sq.NORM_RMS, pre_norm=sq.NORM_LAYER)
    want = sq.block_norm_quant_per_token(x.clone(), res.clone(), **kw)
    before = buf.clone()
    got = sq.block_norm_quant_per_token(x, res, h_out=h, **kw)
    assert got[0] is h
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    h.copy_(before[:, order[2] * (K + gap):order[2] * (K + gap) + K])
    assert torch.equal(buf, before)


def test_block_norm_sums_rows_beside_its_output():
    R, M, K = 900, 400, 512
    buf = torch.randn((R, 2 * K), device="cuda")
    x, h = buf[:, :K], buf[:M, K:]
    rows = torch.randint(-1, R, (M, 3), device="cuda", dtype=torch.int32)
    w = torch.rand((M, 3), device="cuda")
    want = sq.block_norm_quant_per_token(x.clone(), token_row=rows, weights=w, post_norm=sq.NORM_RMS)
    got = sq.block_norm_quant_per_token(x, token_row=rows, weights=w, post_norm=sq.NORM_RMS, h_out=h)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# tokens of many experts
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("fp8", [False, True], ids=["int8", "fp8"])
@pytest.mark.parametrize("M,K,top_k,dtype", [(300, 4096, 8, torch.bfloat16), (40, 8192, 6, torch.bfloat16),
                                             (2600, 2048, 8, torch.bfloat16), (5, 16384, 16, torch.float32),
                                             (33, 9216, 5, torch.float32), (1, 32768, 7, torch.bfloat16)])
def test_block_norm_sums_many_rows(M, K, top_k, dtype, fp8):
    rng = _rng(3, M, K)
    R = M * top_k
    x, res = (_cuda_of(rng.standard_normal((n, K))).to(dtype) for n in (R, M))
    rows = rng.integers(-1, R + 1, (M, top_k)).astype(np.int32)  # some entries name no row
    w = rng.uniform(0, 1, (M, top_k)).astype(np.float32)
    g = rng.uniform(0.5, 1.5, K).astype(np.float32)
    h, q, s = sq.block_norm_quant_per_token(
        x, res, token_row=_cuda_of(rows), weights=_cuda_of(w), post_norm=sq.NORM_RMS, post_gamma=_cuda_of(g),
        residual_scale=0.5, pre_norm=sq.NORM_LAYER, pre_gamma=_cuda_of(g), fp8=fp8)
    hr, dh, y, dy = ref.block_norm(_np64(x), _np64(res), rows, w.astype(np.float64), ("rms", g, None, 1e-5),
                                   None, None, 0.5, ("layer", g, None, 1e-5))
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -23
    assert (np.abs(_np64(h) - hr) <= dh + half * (np.abs(hr) + dh)).all()
    vals = ref.E4M3[q.cpu().numpy()] if fp8 else q.cpu().numpy().astype(np.float64)
    ref.check_codes(vals, _np64(s), y, dy, 448.0 if fp8 else 127.0)


def test_block_norm_without_expert_rows():
    """A part of the experts that got no row: nothing is read, and h is the residual."""
    for M in (3, 5000):
        x = torch.empty((0, 256), device="cuda")
        res = torch.randn((M, 256), device="cuda")
        rows = torch.full((M, 2), -1, dtype=torch.int32, device="cuda")
        w = torch.full((M, 2), float("nan"), device="cuda")
        h, q, s = sq.block_norm_quant_per_token(x, res, token_row=rows, weights=w, post_norm=sq.NORM_RMS)
        want = sq.block_norm_quant_per_token(res)
        for a, b in zip((h, q, s), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("top_k,score", [(1, "softmax"), (4, "sigmoid"), (6, "softmax"), (8, "sigmoid")])
def test_layer_of_tokens_with_several_experts(top_k, score, fmt):
    """Every stage against its 64-bit form on the stage before, for one expert to all of them."""
    layer, act, gamma, Xq, xs, logits, res = _layer(fmt, top_k=top_k, score=score)
    logits[65:] = -float("inf")
    h, q, s = layer.forward(Xq, xs, logits, res, post_norm=sq.NORM_RMS, post_gamma=gamma)
    st = h.stages
    w, e, off, row, tok, bound = ref.route(_np64(logits), top_k, score)
    assert np.array_equal(st["route"].experts.cpu().numpy(), e)
    assert np.array_equal(st["route"].token_row.cpu().numpy(), tok)
    assert (np.abs(_np64(st["route"].weights) - w) <= bound * np.abs(w) + 2.0 ** -126).all()
    fp8, n = fmt == "fp8", int(off[-1])
    val = lambda c: ref.E4M3[c.cpu().numpy()] if fp8 else c.cpu().numpy().astype(np.float64)  # noqa: E731
    a, ha = val(Xq) * _np64(xs)[:, None], val(st["Hq"][:n]) * _np64(st["h_scale"][:n])[:, None]
    wide = val(layer.gate_up_q) * _np64(layer.gate_up_scale)[:, :, None]
    narrow = val(layer.down_q) * _np64(layer.down_scale)[:, :, None]
    gu, y = _np64(st["gate_up"][:n]), _np64(st["down"][:n])
    for ex in range(8):
        sl = slice(off[ex], off[ex + 1])
        for got, left, right in ((gu[sl], a[row[sl]], wide[ex]), (y[sl], ha[sl], narrow[ex])):
            want = left @ right.T
            # accumulation (FP8) and the two scales' roundings, then bf16's half step
            slack = (31 + 8 + 4) * 2.0 ** -23 * (np.abs(left) @ np.abs(right).T)
            assert (np.abs(got - want) <= slack + 2.0 ** -8 * (np.abs(want) + slack)).all()
    g = gamma.cpu().numpy()
    hr, dh, yr, dy = ref.block_norm(y, _np64(res), tok, _np64(st["route"].weights), ("rms", g, None, 1e-5),
                                    pre=("rms", None, None, 1e-5))
    assert (np.abs(_np64(h) - hr) <= dh + 2.0 ** -8 * (np.abs(hr) + dh)).all()
    ref.check_codes(val(q), _np64(s), yr, dy, 448.0 if fp8 else 127.0)


# ---------------------------------------------------------------------------
# the scope of a call
# ---------------------------------------------------------------------------

def test_a_call_leaves_the_current_stream_as_it_was():
    x = torch.randn((40, 64), device="cuda")
    outer, side = torch.cuda.Stream(), torch.cuda.Stream()
    outside = torch.cuda.ExternalStream(side.cuda_stream)
    default = torch.cuda.current_stream()
    want = sq.moe_route(x, 2)
    torch.cuda.synchronize()
    for stream in (None, default, side, outer, outside):
        with torch.cuda.stream(outer):
            got = sq.moe_route(x, 2, stream=stream)
            assert torch.cuda.current_stream() == outer
            with pytest.raises(sq.SQError):  # refused inside the scope
                sq.moe_route(x, 17, stream=stream)
            assert torch.cuda.current_stream() == outer
        assert torch.cuda.current_stream() == default
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
