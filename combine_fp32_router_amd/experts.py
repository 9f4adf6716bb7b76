"""The experts of a layer: two products and the activation between them,
over one contiguous run of rows per expert (the receiver's grouped rows).

    h[p] = act(x[p] W_up[e]^T + b_up[e])
    y[p] = h[p] W_down[e]^T + b_down[e] (+ residual[p])

bf16 rows and weights, fp32 sums; h and y are rounded once each.  With
``train`` the forward call also keeps z = x W_up^T + b_up (bf16), and
``backward`` gives the gradients of the rows, the weights and the biases.
ExpertMLP8 is the same layer with its products in E4M3 codes.
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
        self._through_down(d_out, offsets, n, grads is not None, d_x is not None, stream)
        if grads is not None:
            B.moe_expert_matmul_dw(d_out, self.hidden[:n], offsets, grads.w_down, grads.b_down,
                                   accumulate, stream)
            B.moe_expert_matmul_dw(self.d_preact[:n], x, offsets, grads.w_up, grads.b_up,
                                   accumulate, stream)
        if d_x is not None:
            self._through_up(offsets, n, d_x, stream)

    def _through_down(self, d_out, offsets, n, for_grads, for_x, stream):
        """d_preact from d_out, for the parameters' gradients and for the rows'."""
        B.moe_expert_matmul_dx(d_out, offsets, self.w_down, self.act, self.preact[:n],
                               self.d_preact[:n], stream)

    def _through_up(self, offsets, n, d_x, stream):
        """d_x from d_preact."""
        B.moe_expert_matmul_dx(self.d_preact[:n], offsets, self.w_up, B.MOE_ACT_NONE, None, d_x,
                               stream)


def _capturing(stream: torch.cuda.Stream) -> bool:
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


class ExpertMLP8(ExpertMLP):
    """The experts with E4M3 rows and weights in the products of `forward` and of
    the rows' gradients: a scale for each 1 x 128 of a row and 128 x 128 of a weight,
    fp32 sums.  h goes from one product to the next as codes; the weights'
    gradients are bf16 products, of bf16 rows (`backward` takes x in bf16 also
    where `forward` had it in codes), and a quantisation counts as the identity.

    The codes are those that the weights had when it was made: after a change
    of w_up or w_down, `quantize` takes them again.  Calls on other streams than
    the codes were made on wait for them (but for calls captured into a graph,
    whose replays the caller orders).  `quantize` itself waits for nothing: like any
    other call it is the caller's to order behind calls on other streams."""

    def __init__(self, w_up: torch.Tensor, w_down: torch.Tensor, act: int,
                 b_up: torch.Tensor | None = None, b_down: torch.Tensor | None = None,
                 max_rows: int = 0, train: bool = False, stream=None):
        """`stream`: where the codes are made, behind the current stream's work
        (None: on that itself)."""
        super().__init__(w_up, w_down, act, b_up, b_down, max_rows, train)
        E, H, I, wide, dev = self.E, self.H, self.I, self.wide, self.device
        nbh, nbi = B.code_blocks(H), B.code_blocks(I)

        def coded(codes, scales):
            return (torch.empty(codes, dtype=torch.float8_e4m3fn, device=dev),
                    torch.empty(scales, dtype=torch.float32, device=dev))

        self.up8 = coded((E, wide * I, H), (E, wide, nbi, nbh))
        self.down8 = coded((E, H, I), (E, 1, nbh, nbi))
        self.up8_t = coded((E, H, wide * I), (E, nbh, wide, nbi)) if train else (None, None)
        self.down8_t = coded((E, I, H), (E, nbi, 1, nbh)) if train else (None, None)
        self.x8 = coded((max_rows, H), (max_rows, nbh))  # d_out's, in a backward call
        self.hidden8 = coded((max_rows, I), (max_rows, nbi))
        self.d_preact8 = coded((max_rows, wide * I), (max_rows, wide, nbi)) if train else None
        if not train:
            self.hidden = None
        self._codes_made = None  # event behind the codes' making
        self._behind = set()  # handles of the streams that are behind it
        if dev.type == "cuda":
            if stream is not None:  # the buffers are in the current one's order
                B.stream_of(stream, dev).wait_stream(torch.cuda.current_stream(dev))
            self.quantize(stream)

    def quantize(self, stream=None) -> None:
        """The weights' codes, from w_up and w_down as they are now."""
        B.moe_quant_weights(self.w_up, *self.up8, *self.up8_t, self.wide, stream)
        B.moe_quant_weights(self.w_down, *self.down8, *self.down8_t, 1, stream)
        on = B.stream_of(stream, self.device)
        if not _capturing(on):
            self._codes_made, self._behind = on.record_event(), {on.cuda_stream}

    def _behind_codes(self, stream) -> None:
        """What `stream` is given next waits for the codes."""
        if self._codes_made is None or B.stream_handle(stream, self.device) in self._behind:
            return
        on = B.stream_of(stream, self.device)
        if not _capturing(on):
            on.wait_event(self._codes_made)
            self._behind.add(on.cuda_stream)

    def forward(self, x: torch.Tensor, offsets: torch.Tensor, out: torch.Tensor,
                residual: torch.Tensor | None = None, stream=None,
                scales: torch.Tensor | None = None) -> torch.Tensor:
        """ExpertMLP.forward; with `scales` (fp32 [rows], one a row, or [rows, ceil(H /
        128)]) x is E4M3 codes [rows, H]."""
        n = self._rows(x, "x")
        B._want_bf16(out, (n, self.H), "out")
        h8, hs = self.hidden8[0][:n], self.hidden8[1][:n]
        self.forwards += 1
        self._kept = None
        self._behind_codes(stream)
        if scales is None:
            bf16, (x, scales) = x, (t[:n] for t in self.x8)
            B.moe_quant_rows(bf16, x, scales, offsets, 1, stream)
        B.moe_expert_matmul_fp8(x, scales, offsets, *self.up8, self.b_up, self.act, None,
                                self.hidden[:n] if self.train else None, h8, hs,
                                self.preact[:n] if self.train else None, stream)
        B.moe_expert_matmul_fp8(h8, hs, offsets, *self.down8, self.b_down, B.MOE_ACT_NONE,
                                residual, out, stream=stream)
        self._kept = n
        return out

    def _through_down(self, d_out, offsets, n, for_grads, for_x, stream):
        if not (for_grads or for_x):
            return
        self._behind_codes(stream)
        d8, dz8 = [t[:n] for t in self.x8], [t[:n] for t in self.d_preact8]
        B.moe_quant_rows(d_out, *d8, offsets, 1, stream)
        B.moe_expert_matmul_fp8_dx(*d8, offsets, *self.down8_t, self.act, self.preact[:n],
                                   self.d_preact[:n] if for_grads else None,
                                   *(dz8 if for_x else (None, None)), stream)

    def _through_up(self, offsets, n, d_x, stream):
        B.moe_expert_matmul_fp8_dx(*(t[:n] for t in self.d_preact8), offsets, *self.up8_t,
                                   B.MOE_ACT_NONE, None, d_x, stream=stream)
