"""``GateTrainer``: one training step of a layer's gate, the experts held fixed.

The forward runs the layer's own step-by-step calls and keeps what the
backward needs; the backward gives the gradients of the router's weight and
bias (and, where asked for, of x through the gate and of the experts' output
rows), of a loss on the layer's output plus the balance loss.  All arithmetic
happens in the library's CUDA kernels, on the current stream, with no host
synchronisation."""

from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import binding as B
from .layer import MoELayer


class GateGrads(NamedTuple):
    """What ``GateTrainer.backward`` returns; None where not asked for."""

    dw_g: torch.Tensor                # (d, E) fp32
    dbias: Optional[torch.Tensor]     # (E,) fp32, for a layer with a bias
    dx: Optional[torch.Tensor]        # (T, d) bf16: x's gradient through the gate alone
    dz: Optional[torch.Tensor]        # (T*k, d) bf16: the experts' output rows'
    norm: Optional[torch.Tensor]      # (1,) fp32: of this layer's dw_g and dbias, before clipping


class GateTrainer:
    """Trains the gate of ``layer`` (any expert format, no replica plan).

    ``forward(x)`` returns y and leaves the balance loss in ``loss`` (3,)
    {balance + z, balance, z}, the selections of each expert in ``counts``
    (S, E), the counted tokens in ``tokens`` (S + 2,) and the mean
    probabilities in ``prob_mean`` (S, E); ``backward(dy)`` follows it, any
    number of times, until the next forward.

    A trainer's calls follow one another: on one stream, or on several that the
    caller makes wait for each other.  Its workspaces grow to the largest batch
    and serve all.  A captured step has workspaces of its own (forward and
    backward are captured together), so that graphs can be replayed beside one
    another and beside the trainer's further calls."""

    def __init__(self, layer: MoELayer, balance_coef: float = 1e-2, z_coef: float = 0.0):
        self.layer = layer
        self.balance_coef, self.z_coef = float(balance_coef), float(z_coef)
        self.loss = self.counts = self.tokens = self.prob_mean = None
        self._kept: Optional[dict] = None
        self._ws: dict = {"forward": None, "backward": None}

    def _workspace(self, kind: str, need: int) -> torch.Tensor:
        if need == 0:
            raise B.MoEError(B.MOE_ERR_INVALID_ARG, "GateTrainer")
        captured = torch.cuda.is_current_stream_capturing()
        old = None if captured else self._ws[kind]
        if old is not None and old.numel() >= need:
            return old
        ws = torch.empty(need, dtype=torch.uint8, device=self.layer.w13.device)
        if old is None:
            ws[:64].zero_()  # the header; nothing else is read before it is written
        else:
            ws[:64].copy_(old[:64])  # with the error word
            old.record_stream(torch.cuda.current_stream(old.device))
        if not captured:
            self._ws[kind] = ws
        return ws

    def forward(self, x: torch.Tensor, token_mask: Optional[torch.Tensor] = None,
                seq_offsets: Optional[torch.Tensor] = None) -> torch.Tensor:
        """y = MoE(x) for x (T, d) bf16, and the balance loss over the batch or
        the sequences of ``seq_offsets`` (see moe_balance_loss).  x, the mask
        and the offsets are kept by reference until the next forward."""
        layer = self.layer
        if layer.physical_experts != layer.E:
            raise NotImplementedError("the gate trains without a replica plan")
        T, dev = int(x.shape[0]), layer.w13.device
        S = 1 if seq_offsets is None else len(seq_offsets) - 1
        shape = layer.shape(T)
        ws = self._workspace("forward", B.moe_workspace_size(shape))
        bwd = B._bwd_bytes(T, layer.d, layer.E, layer.k, layer.f, layer.R, S)
        ws_bwd = self._workspace("backward", bwd)
        new = lambda *size, dtype=torch.float32: torch.empty(*size, dtype=dtype, device=dev)  # noqa: E731
        E, k, d = layer.E, layer.k, layer.d
        logits, w = new(T, E), new(T, k)
        idx, row_of = new(T, k, dtype=torch.int32), new(T, k, dtype=torch.int32)
        rows, offsets = new(E, dtype=torch.int32), new(E + 1, dtype=torch.int32)
        perm = new(T * k, dtype=torch.int32)
        x_perm, z = new(T * k, d, dtype=torch.bfloat16), new(T * k, d, dtype=torch.bfloat16)
        y = torch.empty_like(x)
        B.moe_router(x, layer.w_g, layer.bias, logits, shape, ws)
        B.moe_topk(logits, idx, w, shape)
        B.moe_dispatch(idx, x, rows, offsets, perm, row_of, x_perm, shape, ws)
        if layer.fp8:
            ffn = B.moe_ffn_w8a8 if layer.w8a8 else B.moe_ffn_fp8
            ffn(x_perm, offsets, layer.w13, layer.w13_scale, layer.w2, layer.w2_scale, z, shape, ws)
        else:
            B.moe_ffn(x_perm, offsets, layer.w13, layer.w2, z, shape, ws)
        B.moe_combine(z, row_of, w, y, shape)
        loss, counts, mean = new(3), new(S, E, dtype=torch.int32), new(S, E)
        tokens = new(S + 2, dtype=torch.int32)
        B.moe_balance_loss(logits, idx, loss, counts, tokens, shape, ws_bwd,
                           balance_coef=self.balance_coef, z_coef=self.z_coef,
                           token_mask=token_mask, seq_offsets=seq_offsets, prob_mean=mean)
        self.loss, self.counts, self.tokens, self.prob_mean = loss, counts, tokens, mean
        self._kept = dict(x=x, logits=logits, idx=idx, w=w, row_of=row_of, z=z, shape=shape,
                          mask=token_mask, seqs=seq_offsets, ws=ws, ws_bwd=ws_bwd)
        return y

    __call__ = forward

    def backward(self, dy: torch.Tensor, dloss: Optional[torch.Tensor] = None,
                 dx: bool = False, dz: bool = False,
                 max_norm: Optional[float] = None) -> GateGrads:
        """Gradients for the loss whose gradient on y is ``dy`` (T, d) bf16,
        plus ``dloss`` (a (1,) fp32 device tensor, default 1) times the
        balance loss.  ``max_norm``: clips this layer's dw_g and dbias by the norm
        of the two.  For the norm over several layers leave it out and give their
        gradients to one moe_clip_grads.  ``dx`` and ``dz`` end here: the experts'
        own backward, and with it x's gradient through them, is the caller's."""
        if self._kept is None:
            raise RuntimeError("backward needs a forward first")
        q, layer = self._kept, self.layer
        shape, dev = q["shape"], layer.w13.device
        T, E, k, d = shape.T, layer.E, layer.k, layer.d
        ws = q["ws_bwd"]
        dw = torch.empty(T, k, device=dev)
        dzt = torch.empty(T * k, d, dtype=torch.bfloat16, device=dev) if dz else None
        dlogits = torch.empty(T, E, device=dev)
        B.moe_combine_bwd(dy, q["z"], q["row_of"], q["w"], shape, dw=dw, dz=dzt)
        B.moe_gate_bwd(q["logits"], q["idx"], dlogits, shape, ws, w=q["w"], dw=dw,
                       counts=self.counts, tokens=self.tokens, balance_coef=self.balance_coef,
                       z_coef=self.z_coef, dloss=dloss, token_mask=q["mask"],
                       seq_offsets=q["seqs"])
        dw_g = torch.empty_like(layer.w_g)
        dbias = None if layer.bias is None else torch.empty_like(layer.bias)
        dxt = torch.empty_like(q["x"]) if dx else None
        B.moe_router_bwd(q["x"], layer.w_g, dlogits, shape, ws, dw_g=dw_g, dbias=dbias, dx=dxt)
        norm = None
        if max_norm is not None:
            norm = torch.empty(1, device=dev)
            B.moe_clip_grads([dw_g] if dbias is None else [dw_g, dbias], max_norm, norm)
        return GateGrads(dw_g, dbias, dxt, dzt, norm)

    def check(self, stream=None) -> int:
        """Synchronises and returns (and clears) the last step's error word."""
        if self._kept is None:
            return B.MOE_OK
        first = B.moe_check(self._kept["ws"], stream)
        second = B.moe_check(self._kept["ws_bwd"], stream)
        return first if first != B.MOE_OK else second
