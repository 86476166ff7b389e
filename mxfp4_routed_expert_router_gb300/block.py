"""A decoder layer with the operators of the library.

``MoeBlock`` holds the pieces that a decoder layer runs: the norm and the 4-bit
projection in front of attention, attention itself over a paged cache, and behind
it the output projection, the norm, the router, group-limited routing and the
experts.  The residual stream is a float32 [T, H] tensor that is updated in place.  torch
supplies memory and streams only; everything runs on its current stream.
"""
from __future__ import annotations

import dataclasses
from typing import Optional

import torch

from . import binding as B
from .attention import Attention
from .layer import MoeLayer
from .linear import QuantLinear, stream_workspace


@dataclasses.dataclass(frozen=True)
class Routing:
    """How the router's logits choose experts (``moe_route_grouped``)."""

    k: int
    n_groups: int = 1
    k_groups: int = 1
    score: int = B.MOE_SCORE_SIGMOID
    group_score: int = B.MOE_GROUP_TOP2
    renormalize: bool = True
    scale: float = 1.0


class MoeBlock:
    """* in_gain [H], in_proj: the norm and the projection in front of attention (``project_in``)
    * out_proj: attention's output projection (rows of H values), or None when attention's output is added as it is
    * attention, between the two projections (``decode``, ``prompt``: the whole layer), or None for attention of the
      caller's own between ``project_in`` and ``forward``
    * gain [H], router (a [E, H] weight), bias float32 [E] or None, routing, layer: the experts' side (``forward``)

    What does not fit together is refused here or, for the rows of a call, before the call touches the residual stream.
    """

    def __init__(self, layer: MoeLayer, router: QuantLinear, routing: Routing, gain: Optional[torch.Tensor] = None,
                 bias: Optional[torch.Tensor] = None, out_proj: Optional[QuantLinear] = None,
                 in_proj: Optional[QuantLinear] = None, in_gain: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 attention: Optional[Attention] = None):
        H, E, r = layer.cfg.hidden, router.N, routing
        if layer.dense:
            raise B.MoeError(B.MOE_EINVAL, "layer: a layer of routed experts is needed")
        if router.K != H or (out_proj is not None and out_proj.N != H) or (in_proj is not None and in_proj.K != H):
            raise B.MoeError(B.MOE_EINVAL, f"router, out_proj and in_proj: rows of the layer's {H} values are needed")
        if r.k > layer.config.k_max:
            raise B.MoeError(B.MOE_EINVAL, f"routing: k = {r.k} above the layer's {layer.config.k_max}")
        if attention is not None:
            width = attention.n_heads * attention.cache.head_dim
            if in_proj is None or in_proj.N != attention.row:
                raise B.MoeError(B.MOE_EINVAL, f"attention: an in_proj to rows of {attention.row} values is needed")
            if (out_proj.K if out_proj is not None else H) != width:
                raise B.MoeError(B.MOE_EINVAL, f"attention: an out_proj of rows of {width} values is needed")
        if bias is not None and (bias.dtype != torch.float32 or bias.shape != (E,) or not bias.is_contiguous()):
            raise B.MoeError(B.MOE_EINVAL, f"bias: a dense float32 vector of {E} values is needed")
        # (no tokens: the library checks the routing's numbers and enqueues nothing)
        B.moe_route_grouped(None, None, 0, E, r.k, r.n_groups, r.k_groups, r.score, r.group_score, r.renormalize,
                            r.scale, None, None, 0)
        self.layer, self.router, self.routing = layer, router, routing
        self.gain, self.bias, self.out_proj, self.in_proj, self.in_gain = gain, bias, out_proj, in_proj, in_gain
        self.eps, self.attention = eps, attention

    def project_in(self, residual: torch.Tensor) -> torch.Tensor:
        """in_proj of the norm of the residual stream, as bfloat16 rows; the norm's rows are MXFP8 in between."""
        T, H = residual.shape
        q = torch.empty((T, H), dtype=torch.float8_e4m3fn, device=residual.device)
        scales = torch.empty((T, H // 32), dtype=torch.uint8, device=residual.device)
        out = torch.empty((T, self.in_proj.N), dtype=torch.bfloat16, device=residual.device)
        B.moe_add_rmsnorm(residual, None, self.in_gain, self.eps, None, None, q, scales)
        return self.in_proj.forward(q, scales, out=out)

    def _attention(self) -> Attention:
        if self.attention is None:
            raise B.MoeError(B.MOE_EINVAL, "the block has no attention")
        return self.attention

    def decode(self, residual: torch.Tensor, slots: torch.Tensor, positions: Optional[torch.Tensor],
               page_table: torch.Tensor, lens: torch.Tensor) -> torch.Tensor:
        """The whole layer for one new token of each sequence (a row of the residual stream, which it updates in place):
        see ``Attention.decode``."""
        attention = self._attention()
        self._check_stream(residual)
        return self.forward(attention.decode(self.project_in(residual), slots, positions, page_table, lens), residual)

    def prompt(self, residual: torch.Tensor, slots: torch.Tensor, positions: Optional[torch.Tensor],
               offsets: torch.Tensor) -> torch.Tensor:
        """The whole layer for packed prompts (rows of the residual stream, which it updates in place): see
        ``Attention.prompt``."""
        attention = self._attention()
        self._check_stream(residual)
        return self.forward(attention.prompt(self.project_in(residual), slots, positions, offsets), residual)

    def _check_stream(self, residual: torch.Tensor) -> None:
        H = self.layer.cfg.hidden
        if residual.dim() != 2 or residual.shape[1] != H or residual.dtype != torch.float32 or \
                not residual.is_contiguous():  # the experts add to it as a dense float32 [T, H]
            raise B.MoeError(B.MOE_EINVAL, f"residual: dense float32 rows of {H} values are needed, not "
                                           f"{residual.dtype} {tuple(residual.shape)}")

    def forward(self, attn: torch.Tensor, residual: torch.Tensor) -> torch.Tensor:
        """Adds attention's output (bfloat16 rows; out_proj is applied to them) and then the experts' output for
        the norm of the sum to the residual stream, in place."""
        self._check_stream(residual)
        H = self.layer.cfg.hidden
        T, dev, r = residual.shape[0], residual.device, self.routing
        E = self.router.N
        delta = attn if self.out_proj is None else self.out_proj.forward(attn)
        x = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
        B.moe_add_rmsnorm(residual, delta, self.gain, self.eps, residual, x)
        logits = self.router.forward(x)
        ids = torch.empty((T, r.k), dtype=torch.int32, device=dev)
        w = torch.empty((T, r.k), dtype=torch.float32, device=dev)
        B.moe_route_grouped(logits, self.bias, T, E, r.k, r.n_groups, r.k_groups, r.score, r.group_score,
                            r.renormalize, r.scale, ids, w)
        # the stream's workspace, or the captured graph's own, not the layer's: that one is shared by all streams and
        # replaced under a graph when more tokens come
        ws = stream_workspace(max(256, B.moe_workspace_bytes(self.layer.handle, T, r.k)), dev)
        return self.layer.forward_routed(x, ids, w, out=residual, accumulate=True, workspace=ws)
