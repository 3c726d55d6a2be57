"""The operators of a W8A8 mixture-of-experts block: what is measured, and their plain form.

Three operators, run here one pass at a time:

``route``    router logits -> the chosen experts with their weights, and the
             (token, expert) rows sorted by expert;
``grouped``  the 8-bit GEMM of rows sorted by expert with every expert's own
             weight matrix, ragged row counts, dequantised to bf16;
``block``    the end of one block and the start of the next: (weighted sum of
             the experts' rows,) norm, gate, scaled residual, norm, per-token
             INT8 / FP8 codes.

With ``own`` false ``run`` computes them from elementary torch operations in
fp32 (fp64 where a comparison would hang on the last bit); with ``own`` true it
makes the calls of ``w8a8_int8_quantized_norm_b200.sq``.  ``exact`` is the
definition in 64 bits.  Eight-bit codes are returned as the values they stand
for (code x scale), in bf16.
"""
import math

import torch

own = False

FLT_MAX = torch.finfo(torch.float32).max


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _route(name, tokens, experts, top_k, dtype, score, bias, renorm, padded):
    return dict(name=name, op="route", tokens=tokens, experts=experts, top_k=top_k, dtype=dtype,
                score=score, bias=bias, renorm=renorm, padded=padded)


def _grouped(name, tokens, experts, top_k, n, k, fmt, gather, skew, relu):
    return dict(name=name, op="grouped", tokens=tokens, experts=experts, top_k=top_k, n=n, k=k,
                fmt=fmt, gather=gather, skew=skew, relu=relu)


def _block(name, tokens, k, dtype, post, pre, top_k, gate, token_gate, residual, fmt):
    return dict(name=name, op="block", tokens=tokens, k=k, dtype=dtype, post=post, pre=pre,
                top_k=top_k, gate=gate, token_gate=token_gate, residual=residual, fmt=fmt)


def listed():
    return [
        # one token of a decode step over 8 experts: nothing but latency
        _route("route-1x8-top2", 1, 8, 2, "bf16", "softmax", False, True, 0.0),
        # an odd batch of tokens, sigmoid scores chosen with a balancing bias
        _route("route-1999x64-top6-bias", 1999, 64, 6, "f32", "sigmoid", True, True, 0.0),
        # a prefill of 16384 tokens with a padded tail whose logits are masked
        _route("route-16384x128-top8-padded", 16384, 128, 8, "bf16", "softmax", False, False, 0.1),
        # decode, one token: two experts' weights stream through
        _grouped("grouped-int8-1tok-8e-8192x4096", 1, 8, 2, 8192, 4096, "int8", True, 0.0, False),
        # decode, a batch of 32 tokens over 64 experts: a few rows for each
        _grouped("grouped-fp8-32tok-64e-2048x4096", 32, 64, 6, 2048, 4096, "fp8", True, 0.5, False),
        # a mixed batch's down projection: about 100 ragged rows per expert, odd sizes
        _grouped("grouped-int8-777tok-16e-4000x1040", 777, 16, 2, 4000, 1040, "int8", False, 0.5, False),
        # prefill gate/up projection, about 1000 rows per expert
        _grouped("grouped-int8-4096tok-8e-8192x4096", 4096, 8, 2, 8192, 4096, "int8", True, 0.5, False),
        # the largest prefill: 65536 rows over 64 experts of uneven popularity
        _grouped("grouped-fp8-16384tok-64e-4096x4096", 16384, 64, 4, 4096, 4096, "fp8", True, 0.5, False),
        # decode, one token between two blocks with norms on both sides
        _block("block-1x8192-rms-rms", 1, 8192, "bf16", "rms", "rms", 0, False, False, True, "int8"),
        # a decode batch behind the experts: weighted sum of two rows each, a token gate
        _block("block-37x4096-top2-rms", 37, 4096, "bf16", "none", "rms", 2, False, True, True, "int8"),
        # prefill in fp32 with LayerNorms, a channel gate and FP8 codes
        _block("block-4096x9216-layer-fp8", 4096, 9216, "f32", "layer", "layer", 0, True, False, True, "fp8"),
        # prefill behind the experts: 16384 tokens of 8192 channels, norms on both sides
        _block("block-16384x8192-top2-rms-rms", 16384, 8192, "bf16", "rms", "rms", 2, True, False, True, "int8"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "grouped", "grouped", "block"])
    if op == "route":
        experts = _log(rng, 4, 256)
        c = _route("", _log(rng, 1, 16384), experts, min(experts, rng.randint(1, 8)),
                   rng.choice(["bf16", "f32"]), rng.choice(["softmax", "sigmoid"]), False,
                   rng.random() < 0.7, rng.choice([0.0, 0.0, 0.2]))
        c["bias"] = c["score"] == "sigmoid" and rng.random() < 0.5
        while c["tokens"] * experts > 16384 * 128:
            c["tokens"] = max(1, c["tokens"] // 2)
    elif op == "grouped":
        experts = _log(rng, 2, 128)
        c = _grouped("", _log(rng, 1, 16384), experts, min(experts, rng.randint(1, 8)),
                     _log(rng, 64, 8192), 16 * _log(rng, 4, 512), rng.choice(["int8", "fp8"]),
                     rng.random() < 0.6, rng.choice([0.0, 0.5, 1.0]), rng.random() < 0.2)
        while experts * c["n"] * c["k"] > 64 * 4096 * 4096:
            c["n"] = max(64, c["n"] // 2)
            c["k"] = max(64, c["k"] // 32 * 16)
        # the plain form pads every expert to the fullest one
        while c["tokens"] * c["top_k"] * c["n"] * c["k"] * (1 + 3 * c["skew"]) > 65536 * 4096 * 4096 \
                or c["tokens"] * c["top_k"] > 65536:
            c["tokens"] = max(1, c["tokens"] // 2)
    else:
        c = _block("", _log(rng, 1, 16384), 16 * _log(rng, 16, 768), rng.choice(["bf16", "bf16", "f32"]),
                   rng.choice(["none", "rms", "layer"]), rng.choice(["rms", "rms", "layer", "none"]),
                   rng.choice([0, 0, 1, 2, 4]), rng.random() < 0.5, rng.random() < 0.3,
                   rng.random() < 0.8, rng.choice(["int8", "fp8"]))
        while c["tokens"] * c["k"] * max(1, c["top_k"]) * (2 if c["dtype"] == "f32" else 1) > 16384 * 8192 * 2:
            c["tokens"] = max(1, c["tokens"] // 2)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _activations(shape, gen):
    """N(0, 1) with a few channels ten times as large, as a residual stream has."""
    x = torch.randn(shape, generator=gen, device="cuda")
    ch = torch.randint(0, shape[-1], (max(1, shape[-1] // 1000),), generator=gen, device="cuda")
    x[..., ch] *= 10
    return x


def _codes(v, fmt):
    """Per-row absmax codes of fp32 rows: what the program holds as weights and activations."""
    top = 127.0 if fmt == "int8" else 448.0
    scale = v.abs().amax(-1) / top
    q = v / scale.unsqueeze(-1)
    if fmt == "int8":
        return torch.round(q).to(torch.int8), scale
    return q.clamp(-top, top).to(torch.float8_e4m3fn).view(torch.uint8), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dev = "cuda"
    s = dict(case)
    T, k = case["tokens"], case["top_k"]
    if case["op"] == "route":
        E = case["experts"]
        logits = torch.randn((T, E), generator=gen, device=dev) * 1.5
        logits += torch.randn(E, generator=gen, device=dev) * 0.5
        padded = int(T * case["padded"])
        if padded:
            logits[T - padded:] = -math.inf  # the batch's padding: routed nowhere
        s["logits"] = logits.to(_dtype(case["dtype"]))
        s["bias_v"] = torch.randn(E, generator=gen, device=dev) * 0.1 if case["bias"] else None
    elif case["op"] == "grouped":
        E, N, K = case["experts"], case["n"], case["k"]
        pref = torch.randn((T, E), generator=gen, device=dev)
        pref += torch.randn(E, generator=gen, device=dev) * case["skew"]
        chosen = pref.topk(k, dim=1).indices.flatten()
        order = torch.sort(chosen, stable=True).indices
        counts = torch.bincount(chosen, minlength=E)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["capacity"] = int(counts.max())
        if case["gather"]:
            s["row_token"] = (order // k).to(torch.int32)
            s["Xq"], s["x_scale"] = _codes(_activations((T, K), gen), case["fmt"])
        else:
            s["row_token"] = None
            s["Xq"], s["x_scale"] = _codes(_activations((T * k, K), gen), case["fmt"])
        code = torch.int8 if case["fmt"] == "int8" else torch.uint8
        s["Wq"] = torch.empty((E, N, K), dtype=code, device=dev)
        s["w_scale"] = torch.empty((E, N), device=dev)
        for e in range(E):
            s["Wq"][e], s["w_scale"][e] = _codes(torch.randn((N, K), generator=gen, device=dev) * 0.02,
                                                 case["fmt"])
    else:
        K, dt = case["k"], _dtype(case["dtype"])
        R = T * max(1, k)
        s["x"] = _activations((R, K), gen).to(dt)
        s["res"] = (_activations((T, K), gen) * 2).to(dt) if case["residual"] else None
        s["token_row"] = s["weights"] = None
        if k:
            s["token_row"] = torch.randperm(R, generator=gen, device=dev).to(torch.int32).view(T, k)
            s["weights"] = torch.softmax(torch.randn((T, k), generator=gen, device=dev), -1)
        for side in ("post", "pre"):
            kind = case[side]
            s[side + "_gamma"] = torch.rand(K, generator=gen, device=dev) + 0.5 if kind != "none" else None
            s[side + "_beta"] = torch.randn(K, generator=gen, device=dev) * 0.1 if kind == "layer" else None
        s["gate_v"] = torch.rand(K, generator=gen, device=dev) if case["gate"] else None
        s["token_gate_v"] = torch.rand(T, generator=gen, device=dev) if case["token_gate"] else None
        s["residual_scale"] = 0.8
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _values(codes, scale, fmt):
    """The codes as the values they stand for, in bf16."""
    if fmt == "fp8":
        codes = codes.view(torch.float8_e4m3fn).to(torch.bfloat16)
    out = torch.empty(codes.shape, dtype=torch.bfloat16, device=codes.device)
    return torch.mul(codes, scale.unsqueeze(-1), out=out)


def run(state):
    op = state["op"]
    if own:
        from w8a8_int8_quantized_norm_b200 import sq

        if op == "route":
            r = sq.moe_route(state["logits"], state["top_k"], score=state["score"],
                             bias=state["bias_v"], renormalize=state["renorm"], scale=1.0)
            return [r.weights, r.experts, r.offsets, r.row_token, r.token_row]
        if op == "grouped":
            gemm = sq.w8a8_gemm_grouped if state["fmt"] == "int8" else sq.fp8_gemm_grouped
            return gemm(state["Xq"], state["Wq"], state["x_scale"], state["w_scale"],
                        state["offsets"], row_token=state["row_token"],
                        epi="bf16_relu" if state["relu"] else "bf16")
        norms = {"none": sq.NORM_NONE, "rms": sq.NORM_RMS, "layer": sq.NORM_LAYER}
        h, codes, scale = sq.block_norm_quant_per_token(
            state["x"], state["res"], token_row=state["token_row"], weights=state["weights"],
            post_norm=norms[state["post"]], post_gamma=state["post_gamma"],
            post_beta=state["post_beta"], post_eps=1e-5, gate=state["gate_v"],
            token_gate=state["token_gate_v"], residual_scale=state["residual_scale"],
            pre_norm=norms[state["pre"]], pre_gamma=state["pre_gamma"],
            pre_beta=state["pre_beta"], pre_eps=1e-5, fp8=state["fmt"] == "fp8")
        return [h, _values(codes, scale, state["fmt"]), scale]
    if op == "route":
        return _plain_route(state)
    if op == "grouped":
        return _plain_grouped(state)
    return _plain_block(state)


def _plain_route(s):
    k, E = s["top_k"], s["experts"]
    logits = s["logits"].float()
    T = logits.shape[0]
    ok = ~torch.isnan(logits) & (logits != -math.inf)
    logits = torch.where(ok, logits.clamp(max=FLT_MAX), -math.inf)
    if s["bias_v"] is not None:
        # two scores next to each other must not swap for a rounding: 64 bits
        key = 1.0 / (1.0 + torch.exp(-logits.double())) + s["bias_v"].double()
        key = torch.where(ok, key, -math.inf)
    else:
        key = logits  # both scores rise with the logit
    order = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    live = torch.gather(ok, 1, order)
    if s["score"] == "softmax":
        top = torch.where(ok, logits, -FLT_MAX).amax(1, keepdim=True)
        p = torch.where(ok, torch.exp(logits - top), 0.0)
        total = p.sum(1, keepdim=True)
    else:
        p = torch.where(ok, 1.0 / (1.0 + torch.exp(-logits)), 0.0)
        total = torch.ones((T, 1), device=p.device)
    chosen = torch.gather(p, 1, order) * live
    if s["renorm"]:
        total = chosen.sum(1, keepdim=True)
    weights = torch.where(total > 0, chosen / total, 0.0)
    experts = torch.where(live, order, -1).to(torch.int32)
    flat = torch.where(live, order, E).flatten()
    by_expert, at = torch.sort(flat, stable=True)
    offsets = torch.searchsorted(by_expert, torch.arange(E + 1, device=flat.device)).to(torch.int32)
    in_use = by_expert < E
    row_token = torch.where(in_use, at // k, -1).to(torch.int32)
    rank = torch.empty_like(at)
    rank[at] = torch.arange(T * k, device=at.device)
    token_row = torch.where(live.flatten(), rank, -1).to(torch.int32).view(T, k)
    return [weights, experts, offsets, row_token, token_row]


def _decoded(codes, fmt):
    return codes.float() if fmt == "int8" else codes.view(torch.float8_e4m3fn).float()


def _plain_grouped(s):
    """Every expert's rows padded to the fullest expert's, one batched fp32 product (the INT8
    sums of these inputs stay far below 2^24, where fp32 holds every integer)."""
    off = s["offsets"].long()
    R = s["tokens"] * s["top_k"]
    dev = off.device
    slot = torch.arange(s["capacity"], device=dev)
    rows = (off[:-1, None] + slot).clamp(max=R - 1)
    src = rows if s["row_token"] is None else s["row_token"].long()[rows]
    acc = torch.bmm(_decoded(s["Xq"][src], s["fmt"]), _decoded(s["Wq"], s["fmt"]).transpose(1, 2))
    acc = acc * s["x_scale"][src].unsqueeze(-1) * s["w_scale"].unsqueeze(1)
    if s["relu"]:
        acc = acc.clamp(min=0)
    r = torch.arange(R, device=dev)
    e = torch.searchsorted(off, r, right=True) - 1
    return acc.to(torch.bfloat16)[e, r - off[e]]


def _norm(v, kind, gamma, beta, eps):
    if kind == "none":
        return v
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    v = v / torch.sqrt(v.square().mean(-1, keepdim=True) + eps) * gamma
    return v if beta is None else v + beta


def _plain_block(s):
    x = s["x"].float()
    if s["top_k"]:
        x = (x[s["token_row"].long()] * s["weights"].unsqueeze(-1)).sum(1)
    h = _norm(x, s["post"], s["post_gamma"], s["post_beta"], 1e-5)
    if s["gate_v"] is not None:
        h = h * s["gate_v"]
    if s["token_gate_v"] is not None:
        h = h * s["token_gate_v"].unsqueeze(1)
    if s["res"] is not None:
        h = s["res"].float() * s["residual_scale"] + h
    y = _norm(h, s["pre"], s["pre_gamma"], s["pre_beta"], 1e-5)
    top = 127.0 if s["fmt"] == "int8" else 448.0
    scale = y.abs().amax(-1) / top
    q = torch.where(scale.unsqueeze(-1) > 0, y / scale.unsqueeze(-1), 0.0).clamp(-top, top)
    codes = torch.round(q).to(torch.int8) if s["fmt"] == "int8" else \
        q.to(torch.float8_e4m3fn).view(torch.uint8)
    return [h.to(s["x"].dtype), _values(codes, scale, s["fmt"]), scale]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    T, k = case["tokens"], case["top_k"]
    if case["op"] == "route":
        E = case["experts"]
        es = 2 if case["dtype"] == "bf16" else 4
        # logits in; weights, experts and both row maps out, the offsets
        return {"bytes": T * E * es + 16 * T * k + 4 * (E + 1), "flops": 4 * T * E}
    if case["op"] == "grouped":
        E, N, K, R = case["experts"], case["n"], case["k"], T * k
        active = E * (1 - (1 - k / E) ** T)  # experts that get a row, at even popularity
        rows = T if case["gather"] else R
        return {"bytes": active * (N * K + 4 * N) + rows * (K + 4) + 4 * R + 4 * (E + 1) + 2 * R * N,
                "flops": 2 * R * N * K}
    K = case["k"]
    es = 2 if case["dtype"] == "bf16" else 4
    vectors = sum({"none": 0, "rms": 1, "layer": 2}[case[n]] for n in ("post", "pre")) + case["gate"]
    moved = T * K * (es * max(1, k) + es * case["residual"] + es + 1)
    return {"bytes": moved + 4 * K * vectors + 4 * T + 8 * T * k, "flops": 12 * T * K}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(s)
    if case["op"] == "grouped":
        return _exact_grouped(s)
    return _exact_block(s)


def _exact_route(s):
    """k rounds of taking the largest key that is left, the first of equal ones."""
    x = s["logits"].double()
    T, E = x.shape
    ok = torch.isfinite(x)
    score = torch.sigmoid(x) if s["score"] == "sigmoid" else \
        torch.nan_to_num(torch.softmax(torch.where(ok, x, -math.inf), 1))
    key = score + s["bias_v"].double() if s["bias_v"] is not None else x
    key = torch.where(ok, key, -math.inf)
    index = torch.arange(E, device=x.device).expand(T, E)
    picks = []
    for _ in range(s["top_k"]):
        best = key.amax(1, keepdim=True)
        first = torch.where(key == best, index, E).amin(1)
        some = best[:, 0] > -math.inf
        picks.append(torch.where(some, score.gather(1, first[:, None])[:, 0], 0.0))
        key = key.scatter(1, first[:, None], -math.inf)
    w = torch.stack(picks, 1)
    if s["renorm"]:
        w = torch.nan_to_num(w / w.sum(1, keepdim=True))
    return [w, None, None, None, None]


def _exact_grouped(s):
    wide = (lambda c: c.double()) if s["fmt"] == "int8" else \
        (lambda c: c.view(torch.float8_e4m3fn).double())
    off = s["offsets"].tolist()
    out = torch.zeros((off[-1], s["n"]), dtype=torch.float64, device="cuda")
    for e in range(s["experts"]):
        r = torch.arange(off[e], off[e + 1], device="cuda")
        src = r if s["row_token"] is None else s["row_token"][r].long()
        x = wide(s["Xq"][src]) * s["x_scale"][src].double()[:, None]
        out[off[e]:off[e + 1]] = x @ (wide(s["Wq"][e]) * s["w_scale"][e].double()[:, None]).T
    return out.relu() if s["relu"] else out


def _exact_block(s):
    x = s["x"].double()
    if s["top_k"]:
        x = sum(x[s["token_row"][:, j].long()] * s["weights"][:, j, None].double()
                for j in range(s["top_k"]))

    def norm(v, kind, side):
        if kind == "none":
            return v
        mu = v.mean(-1, keepdim=True) if kind == "layer" else 0.0
        out = (v - mu) * ((v - mu) ** 2).mean(-1, keepdim=True).add(1e-5).rsqrt() * s[side + "_gamma"].double()
        return out + s[side + "_beta"].double() if kind == "layer" else out

    h = norm(x, s["post"], "post")
    h = h * s["gate_v"].double() if s["gate_v"] is not None else h
    h = h * s["token_gate_v"].double()[:, None] if s["token_gate_v"] is not None else h
    h = h + s["residual_scale"] * s["res"].double() if s["res"] is not None else h
    y = norm(h, s["pre"], "pre")
    step = y.abs().amax(-1, keepdim=True) / (127.0 if s["fmt"] == "int8" else 448.0)
    t = torch.nan_to_num(y / step)
    if s["fmt"] == "int8":
        unit = 1.0
    else:  # three mantissa bits, exponents down to -6
        unit = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6))) - 3)
    return [h, torch.round(t / unit) * unit * step, step[:, 0]]
