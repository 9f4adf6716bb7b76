"""The experts of a layer: two products and the activation between them,
over one contiguous run of rows per expert (the receiver's grouped rows).

    h[p] = act(x[p] W_up[e]^T + b_up[e])
    y[p] = h[p] W_down[e]^T + b_down[e] (+ residual[p])

bf16 rows and weights, fp32 sums; h and y are rounded once each.  With
``train`` the forward call also keeps z = x W_up^T + b_up (bf16), and
``backward`` gives the gradients of the rows, the weights and the biases.
All arithmetic runs in the HIP library; this module allocates (torch) and
orders launches.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import binding as B


class ExpertGrads(NamedTuple):
    """Gradients of an ExpertMLP's parameters, in their shapes."""
    w_up: torch.Tensor                 # fp32 or bf16
    w_down: torch.Tensor
    b_up: torch.Tensor | None = None   # fp32
    b_down: torch.Tensor | None = None


class ExpertMLP:
    """w_up bf16 [E, I, H] (MOE_ACT_SWIGLU: [E, 2I, H], an expert's I gate
    rows, then its I up rows), w_down bf16 [E, H, I], biases fp32 or None;
    buffers for max_rows rows.

    The buffers hold one forward call: every other one, of another batch or
    layer too, takes their place.  `forwards` counts the calls, so that a
    backward call can say which one it belongs to.  (A replayed graph counts
    nothing.)"""

    def __init__(self, w_up: torch.Tensor, w_down: torch.Tensor, act: int,
                 b_up: torch.Tensor | None = None, b_down: torch.Tensor | None = None,
                 max_rows: int = 0, train: bool = False):
        if w_up.dim() != 3 or w_down.dim() != 3:
            raise ValueError("weights must be [E, I, H] and [E, H, I]")
        self.wide = 2 if act == B.MOE_ACT_SWIGLU else 1
        self.E, self.H, self.I = w_down.shape
        B._want_bf16(w_up, (self.E, self.wide * self.I, self.H), "w_up")
        B._want_bf16(w_down, (self.E, self.H, self.I), "w_down")
        for b, n, name in ((b_up, self.wide * self.I, "b_up"), (b_down, self.H, "b_down")):
            if b is not None:
                B._want(b, torch.float32, name)
                if b.numel() != self.E * n:
                    raise ValueError(f"{name} must hold {self.E}*{n} values")
        self.w_up, self.w_down, self.act = w_up, w_down, act
        self.b_up, self.b_down = b_up, b_down
        self.max_rows, self.train = max_rows, train
        self.device = w_up.device

        def rows(n):
            return torch.empty((max_rows, n), dtype=torch.bfloat16, device=self.device)

        self.hidden = rows(self.I)
        self.preact = rows(self.wide * self.I) if train else None
        self.d_preact = rows(self.wide * self.I) if train else None
        self.forwards = 0
        self._kept = None  # rows of the forward call that the buffers hold

    def _rows(self, t: torch.Tensor, name: str) -> int:
        if t.dim() != 2 or t.shape[1] != self.H:
            raise ValueError(f"{name} must be [rows, {self.H}]")
        if t.shape[0] > self.max_rows:
            raise ValueError(f"{name}: {t.shape[0]} rows, buffers for {self.max_rows}")
        return t.shape[0]

    def forward(self, x: torch.Tensor, offsets: torch.Tensor, out: torch.Tensor,
                residual: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """x bf16 [rows, H] in runs of offsets int32 [E+1] -> out bf16
        [rows, H]; rows of no run are not written."""
        n = self._rows(x, "x")
        hidden = self.hidden[:n]
        self.forwards += 1
        self._kept = None
        B.moe_expert_matmul(x, offsets, self.w_up, self.b_up, self.act, None, hidden,
                            self.preact[:n] if self.train else None, stream)
        B.moe_expert_matmul(hidden, offsets, self.w_down, self.b_down, B.MOE_ACT_NONE, residual,
                            out, None, stream)
        self._kept = n
        return out

    def alloc_grads(self, dtype=torch.float32) -> ExpertGrads:
        def f32(b):
            return None if b is None else torch.empty_like(b)

        return ExpertGrads(torch.empty_like(self.w_up, dtype=dtype),
                           torch.empty_like(self.w_down, dtype=dtype), f32(self.b_up),
                           f32(self.b_down))

    def backward(self, d_out: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor,
                 d_x: torch.Tensor | None, grads: ExpertGrads | None, accumulate: bool = False,
                 stream=None, forward: int | None = None) -> None:
        """Gradients of the last forward(x, offsets, ...) from d_out bf16
        [rows, H]: d_x bf16 [rows, H] (may be d_out itself; None: not
        wanted) and grads (None: not wanted), which `accumulate` adds to.
        (A residual's gradient is d_out itself.)  `forward`, what `forwards`
        was after the call meant, refuses if another has run since."""
        if not self.train:
            raise ValueError("backward needs train=True")
        n = self._rows(x, "x")
        if self._kept is None:
            raise ValueError("backward before a whole forward")
        if self._kept != n:
            raise ValueError(f"backward of {n} rows, the last forward had {self._kept}")
        if forward is not None and forward != self.forwards:
            raise ValueError("the experts have run again since that forward")
        hidden, dz = self.hidden[:n], self.d_preact[:n]
        B.moe_expert_matmul_dx(d_out, offsets, self.w_down, self.act, self.preact[:n], dz, stream)
        if grads is not None:
            B.moe_expert_matmul_dw(d_out, hidden, offsets, grads.w_down, grads.b_down, accumulate,
                                   stream)
            B.moe_expert_matmul_dw(dz, x, offsets, grads.w_up, grads.b_up, accumulate, stream)
        if d_x is not None:
            B.moe_expert_matmul_dx(dz, offsets, self.w_up, B.MOE_ACT_NONE, None, d_x, stream)
