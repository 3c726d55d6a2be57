"""The expert MLP of a block in W8A8, from the library's calls.

The source pages treat dense blocks; their scheme carries over unchanged
("SmoothQuant, in depth" -- "Where the scales go in a decoder block",
"Granularity"): every expert's gate/up projection reads one norm, so they share
one smoothing factor folded into it; the down projections' input SiLU(gate) *
up has no norm in front and is quantised per token without smoothing; weights
have one scale per output channel of each expert.

A layer is six calls: the router's choice and the rows sorted by expert, the
grouped gate/up GEMM that gathers its tokens, SiLU * up with its codes, the
grouped down GEMM, and the block call that sums each token's rows and goes on
to the next block's codes.  Every step runs in libsq.so; this module sequences
the calls and owns the prepared weights.
"""
from __future__ import annotations

import weakref
from typing import Optional

import torch

from . import sq

FORMATS = ("int8", "fp8")


class Stages(dict):
    """The stages of one pass: route, gate_up, Hq, h_scale, down."""


class MoELayer:
    """Experts with gate_up [E, 2 I, H] (gate rows first) and down [E, H, I],
    bf16 or fp32 on the device.  ``prepare`` smooths and quantises them once;
    ``forward`` runs a batch of tokens.

    The layer holds no pass's tensors.  A pass's stages are ``h.stages`` of the h
    it returned and are freed with it; ``layer.stages`` finds those of the
    layer's last pass while they live (else None).  With ``keep_stages`` False
    they are freed within the pass, each as soon as the next one is computed."""

    def __init__(self, gate_up: torch.Tensor, down: torch.Tensor, top_k: int,
                 score: str = "softmax", bias: Optional[torch.Tensor] = None,
                 renormalize: bool = True, scale: float = 1.0, fmt: str = "int8",
                 keep_stages: bool = True):
        E, I2, H = gate_up.shape
        if I2 % 2 or tuple(down.shape) != (E, H, I2 // 2):
            raise ValueError("gate_up must be [E, 2 I, H] and down [E, H, I]")
        if fmt not in FORMATS:
            raise ValueError("fmt must be one of %s" % (FORMATS,))
        if not gate_up.is_contiguous() or not down.is_contiguous():
            raise ValueError("gate_up and down must be contiguous")
        self.gate_up, self.down = gate_up, down
        self.E, self.I, self.H = E, I2 // 2, H
        self.top_k, self.score, self.bias = top_k, score, bias
        self.renormalize, self.scale, self.fmt = renormalize, float(scale), fmt
        self.s = self.gamma = self.beta = None
        self.keep_stages, self._last = keep_stages, None

    @property
    def stages(self) -> Optional[Stages]:
        return self._last() if self._last is not None else None

    def __getstate__(self):  # a copied or saved layer has run no pass
        return dict(self.__dict__, _last=None)

    def prepare(self, act_max: Optional[torch.Tensor] = None, alpha: float = 0.5, gamma=None,
                beta=None, stream=None) -> "MoELayer":
        """Quantise the experts.  With ``act_max`` [H] (sq.calibrate_absmax of the
        norm in front) the gate/up projections are smoothed with one shared s,
        and ``self.gamma`` / ``self.beta`` become that norm's folded parameters;
        without it they are the given ones."""
        wide = self.gate_up.view(self.E * 2 * self.I, self.H)
        narrow = self.down.view(self.E * self.H, self.I)
        self.s, self.gamma, self.beta = None, gamma, beta
        if act_max is not None:
            self.s, self.gamma, self.beta = sq.compute_smooth_scales(
                act_max, [wide], alpha, gamma=gamma, beta=beta, stream=stream)
        quant = sq.smooth_quantize_weights if self.fmt == "int8" else \
            sq.smooth_quantize_weights_fp8
        q, sc = quant(wide, self.s, stream=stream)
        self.gate_up_q = q.view(self.E, 2 * self.I, self.H)
        self.gate_up_scale = sc.view(self.E, 2 * self.I)
        q, sc = quant(narrow, None, stream=stream)
        self.down_q = q.view(self.E, self.H, self.I)
        self.down_scale = sc.view(self.E, self.H)
        return self

    def forward(self, Xq: torch.Tensor, x_scale: torch.Tensor, logits: torch.Tensor,
                residual: Optional[torch.Tensor] = None, stream=None, **block):
        """Tokens' codes Xq [T, H] with x_scale [T] (the norm with ``self.gamma``
        / ``self.beta``) and the router's logits [T, E] -> (h, codes, scales) of
        sq.block_norm_quant_per_token: h = residual_scale * residual + post_norm(sum
        of the experts) * gate ..., and the next norm's codes.  ``block`` are that
        call's norms, gates and outputs.  The stages are ``h.stages``."""
        if Xq.dim() != 2 or tuple(logits.shape) != (Xq.shape[0], self.E):
            raise ValueError("logits must be [T, E] = [%d, %d] for Xq [T, H]"
                             % (Xq.shape[0], self.E))
        gemm = sq.w8a8_gemm_grouped if self.fmt == "int8" else sq.fp8_gemm_grouped
        r = sq.moe_route(logits, self.top_k, self.score, self.bias, self.renormalize, self.scale,
                         stream=stream)
        stages = Stages(route=r)
        gu = gemm(Xq, self.gate_up_q, x_scale, self.gate_up_scale, r.offsets,
                  row_token=r.row_token, stream=stream)
        # rows behind the last expert's hold no values; theirs are never read
        hq, hs = sq.silu_mul_quant_per_token(gu, stream=stream, fp8=self.fmt == "fp8")
        if self.keep_stages:
            stages.update(gate_up=gu, Hq=hq, h_scale=hs)
        del gu
        y = gemm(hq, self.down_q, hs, self.down_scale, r.offsets, stream=stream)
        if self.keep_stages:
            stages.update(down=y)
        del hq, hs
        out = sq.block_norm_quant_per_token(y, residual, token_row=r.token_row, weights=r.weights,
                                            fp8=self.fmt == "fp8", stream=stream, **block)
        self._last = None
        if self.keep_stages:
            out[0].stages = stages
            self._last = weakref.ref(stages)
        return out
