"""A decoder's mixture-of-experts block around the routed int4 experts.

``MoeBlock`` chains the library's operators for serving, with the low-rank
adapters of many requests beside the latent projections:

    idx, w = route_grouped(h, ...)                     softmax or sigmoid, groups
    u      = adapter_linear(h, lat_down, ids)          (latent blocks)
    y      = combine(expert_ffn(dispatch(idx, u)), w)
    y      = adapter_linear(rmsnorm(y), lat_up, ids)   (latent blocks)
    y     += shared_expert(h)                          (with shared_* weights)
    x, h   = block_norm(y, x, ...)                     norm, gate, residual, next norm

With ``few_tokens`` a call of at most 32 tokens, with 1.5 tokens to an expert or fewer on
average, runs dispatch, experts and combine as one operator, ``experts_few``.  It reads an
expert's weights once for every two tokens; the other path, once for 16.  Whole layers,
this way and the other, us: 8 of 384 experts of 7168 x 2048, 1 token 53 and 97, 24 tokens
672 and 752; 8 of 128 experts of 4096 x 1536, 24 tokens 277 and 280, 32 tokens 351 and 307;
2 of 8 experts of 4096 x 14336, 8 tokens 186 and 202, 16 tokens 302 and 209.

The latent path is the one of the "Kimi K3 latent up-projection" page
(KimiSparseMoeBlock.forward: router on the full width, down-projection, experts,
norm, up-projection); groups, adapters, the norm after the block and its gate
are the caller's choice and on none of the pages.
"""
from __future__ import annotations

from typing import Dict, Optional, Tuple

import torch

from . import capi

# the low-rank weights of one projection: A [adapters, R, K], B [adapters, N, R]
# and the adapters' scales (None: 1)
Adapters = Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]


class MoeBlock:
    """Weights and options of one block.

    weights   router_w fp32 [E, H], the stacked int4 experts (gate / up / down
              packed and scale), optionally router_bias fp32 [E]; for a latent
              block lat_down bf16 [L, H], lat_up bf16 [H, L] and optionally
              lat_norm bf16 [L]; for a shared expert shared_gate and shared_up
              bf16 [I, H] and shared_down bf16 [H, I]; router_w_terms (from
              ``router_prepare``; made here where it is missing).  Other names
              are refused
    k, ...    routing options of ``route_grouped``
    adapters  {"lat_down": (A, B, scale), "lat_up": ...}: either, or none
    post_gain, next_gain, gate (a gain per channel, [H]), gate_sigmoid,
    residual_scale, eps: options of ``block_norm``
    few_tokens  calls of few tokens (above) through ``experts_few`` (the expert outputs
              are then summed unrounded, so the bits differ from the other path's)
    """

    def __init__(self, weights: Dict[str, torch.Tensor], k: int, *, score: str = "sigmoid",
                 groups: int = 1, topk_groups: Optional[int] = None, group_score: str = "top2",
                 renorm: bool = True, route_scale: float = 1.0,
                 adapters: Optional[Dict[str, Adapters]] = None,
                 post_gain: Optional[torch.Tensor] = None,
                 next_gain: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                 gate_sigmoid: bool = False, residual_scale: float = 1.0, eps: float = 1e-6,
                 few_tokens: bool = False):
        extra = set(weights) - {n for n, _ in capi.MoeWeights._fields_}
        if extra:
            raise ValueError(f"unknown weight names: {sorted(extra)}")
        for name in ("router_w", *capi.EXPERT_NAMES):
            if name not in weights:
                raise ValueError(f"{name} is required")
        self.experts = {n: weights[n] for n in capi.EXPERT_NAMES}
        self.weights = weights = {n: t for n, t in weights.items() if t is not None}
        self.latent = "lat_down" in weights
        if self.latent != ("lat_up" in weights):
            raise ValueError("lat_down and lat_up come together")
        if "lat_norm" in weights and not self.latent:
            raise ValueError("lat_norm belongs to a latent block (lat_down, lat_up)")
        shared = [weights.get(n) for n in ("shared_gate", "shared_up", "shared_down")]
        if len({t is None for t in shared}) > 1:
            raise ValueError("shared_gate, shared_up and shared_down come together")
        self.shared = None if shared[0] is None else shared
        self.adapters = dict(adapters or {})
        unknown = set(self.adapters) - ({"lat_down", "lat_up"} if self.latent else set())
        if unknown:
            raise ValueError(f"no projection for the adapters of {sorted(unknown)}")
        self.E = weights["router_w"].shape[0]
        self.routing = dict(k=k, bias=weights.get("router_bias"), score=score, groups=groups,
                            topk_groups=topk_groups, group_score=group_score, renorm=renorm,
                            scale=route_scale)
        self.norm = dict(post_gain=post_gain, pre_gain=next_gain, gate=gate,
                         gate_sigmoid=gate_sigmoid, scale=residual_scale, eps=eps)
        self.eps = eps
        self.few_tokens = few_tokens
        # the router weight's bf16 terms, for calls of 512 tokens or more
        self.w_terms = weights.get("router_w_terms")
        if self.w_terms is None:
            self.w_terms = capi.router_prepare(weights["router_w"])

    def route(self, h: torch.Tensor):
        """(topk_idx, topk_w) of the block's input h bf16 [T, H]."""
        return capi.route_grouped(h, self.weights["router_w"], w_terms=self.w_terms,
                                  **self.routing)

    def _project(self, name: str, x: torch.Tensor, ids: Optional[torch.Tensor]) -> torch.Tensor:
        if ids is None or name not in self.adapters:
            return capi.linear_bf16(x, self.weights[name])
        a, b, scale = self.adapters[name]
        return capi.adapter_linear(x, self.weights[name], a, b, ids, scale=scale)

    def forward(self, x: torch.Tensor, h: torch.Tensor, ids: Optional[torch.Tensor] = None,
                x_out: Optional[torch.Tensor] = None):
        """(x', h'): the new residual stream and the next block's input (None
        without next_gain) from the stream x bf16 or fp32 [T, H] and the normed
        input h bf16 [T, H].  ids int32 [T]: each token's adapter (-1: none;
        None: no adapters).  x_out may be x (in place)."""
        idx, w = self.route(h)
        u = self._project("lat_down", h, ids) if self.latent else h
        if (self.few_tokens and h.shape[0] <= capi.FEW_TOKENS
                and 2 * idx.numel() <= 3 * self.E):
            y = capi.experts_few(idx, w, u, self.experts)
        else:
            d = capi.dispatch(idx, u, self.E, pairs=True)
            y = capi.expert_ffn(d["x_sorted"], None, d["offsets"], self.experts, pairs=True,
                                max_rows_per_expert=h.shape[0])
            y = capi.combine(y, d["inv_row"], w)
        if self.latent:
            if "lat_norm" in self.weights:
                y = capi.rmsnorm(y, self.weights["lat_norm"], self.eps)
            y = self._project("lat_up", y, ids)
        if self.shared is not None:
            y = capi.shared_expert(h, *self.shared, out=y)
        return capi.block_norm(y, x, x_out=x_out, **self.norm)
