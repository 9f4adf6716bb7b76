"""All R ranks of one expert-parallel group on one device.

The batch is cut into R consecutive token shards, shard s playing source
rank s.  Each rank routes, lays out and packs its shard into its own flat
send buffer (one segment per destination rank, NCCL EP article s3.3); the
payload all-to-all becomes a block transpose into the ranks' receive
buffers (``moe_exchange_blocks``, a stand-in for the collective); each
receiver computes its row maps (``moe_recv_layout``) and regroups its rows
into one run per expert (``moe_recv_regroup``),
the experts run (an ``ExpertMLP`` over all E experts, or the test stand-in
y = x*(1+e/8)), the rows go back to arrival order (``moe_recv_ungroup``) and
through the reverse exchange, and every source combines its own tokens
(Perseus write-up s1.1: gate, dispatch, experts, combine).

An ``ExpertMLP`` takes and gives bf16 rows.  Between it and a quantised
payload the regroup dequantises in the same pass, as a combine of one slot of
weight 1 over the row map (each row rounded once to bf16), and the ungroup
quantises, as a pack of one slot.

With ``train=True`` experts, ``backward`` runs the last ``run``'s layer the
other way: the combine's gradient at every source, the exchange, the regroup,
the experts' gradients, the ungroup, the exchange back, a combine with weights
1 (the pack's gradient), and the router's gradient with the balance loss.
Gradient rows travel as bf16 whatever the payload, and a payload's
quantisation counts as the identity.

Every buffer holds all ranks end to end, so one launch of each kernel does
the work of all R ranks.  With capacity off, the grouped buffer equals the
single-source dispatch of the whole batch, and the output equals the
chunked layer's with one chunk per shard.  All arithmetic runs in the HIP
library; this module allocates (torch) and orders launches.
"""
from __future__ import annotations

import functools

import torch

from . import binding as B
from . import harness as HN
from .driver import KernelTimer, chunk_capacity, chunk_ranges
from .experts import ExpertGrads, ExpertMLP


def _group_device(call):
    """`call` with the group's device current: a null stream is its own."""
    @functools.wraps(call)
    def on_device(self, *args, **kwargs):
        if self.device.type != "cuda":  # refused further in
            return call(self, *args, **kwargs)
        with torch.cuda.device(self.device):
            return call(self, *args, **kwargs)

    return on_device


class EPGroup:
    def __init__(self, T: int, H: int, E: int, k: int, R: int, standin: bool = True,
                 device="cuda", experts: ExpertMLP | None = None):
        self.T, self.H, self.E, self.k, self.R = T, H, E, k, R
        # `cuda` is the device that is current now, whichever is in a later call
        self.device = torch.empty(0, device=device).device
        self.experts = experts
        self.standin = standin = standin and experts is None
        self.bounds = chunk_ranges(T, R)
        self.Ts = max((b - a for a, b in self.bounds), default=0)
        self.source_rows = self.Ts * k
        self.max_rows = R * self.source_rows
        stride = max(B.moe_row_bytes(H, q) for q in (0, 1, 2, 3))
        rows = max(self.max_rows, 1)
        dev = self.device
        self.idx = torch.empty((max(T, 1), k), dtype=torch.int32, device=dev)
        self.w = torch.empty((max(T, 1), k), dtype=torch.float32, device=dev)
        self.lay = B.alloc_layout_chunks(T, max(self.Ts, 1), E, k, R, dev, R)
        # sources past the last token (T < R) have no layout launch: zero rows
        self.lay.expert_offsets.zero_()
        self.src_offsets = self.lay.expert_offsets[:R]
        self.views = [B.layout_view(self.lay, s, T) for s in range(R)]
        self.rl = B.alloc_recv_layout(E, R, self.max_rows, dev)
        self.send = torch.empty((rows, stride), dtype=torch.uint8, device=dev)
        self.recv = torch.empty_like(self.send)
        self.grouped = torch.empty_like(self.send)
        self.ret = torch.empty_like(self.send) if standin else None
        # one fp32 scale per row of each buffer (quantised payloads)
        scales = lambda: torch.empty(rows, dtype=torch.float32, device=dev)
        self.send_scales, self.recv_scales, self.grouped_scales = scales(), scales(), scales()
        self.ret_scales = scales() if standin else None
        self._caps = {}
        self._last = None  # what backward needs to know of the last whole run
        self._forward = None  # the experts' call of that run
        if experts is not None:
            if (experts.E, experts.H) != (E, H):
                raise ValueError(f"experts [{experts.E}, {experts.H}] in a group of [{E}, {H}]")
            if experts.max_rows < self.max_rows:
                raise ValueError(f"experts' buffers hold {experts.max_rows} of {self.max_rows} rows")

            def rows16():
                return torch.empty((self.max_rows, H), dtype=torch.bfloat16, device=dev)

            self.ones = torch.ones(rows, dtype=torch.float32, device=dev)
            self.expert_in, self.expert_out = rows16(), rows16()
            if experts.train:
                self.d_send, self.d_recv, self.d_rows = rows16(), rows16(), rows16()
                self.d_w = torch.empty((max(T, 1), k), dtype=torch.float32, device=dev)

    def _source_caps(self, factor):
        key = str(factor)
        if key not in self._caps:
            caps = [chunk_capacity(t1 - t0, self.k, self.E, factor) for t0, t1 in self.bounds]
            caps += [0] * (self.lay.expert_offsets.shape[0] - len(caps))
            self._caps[key] = torch.tensor(caps, dtype=torch.int32, device=self.device)
        return self._caps[key]

    def send_rows(self, s: int, quant: int) -> torch.Tensor:
        """Source s's send buffer: rows are dense rows of the payload's
        stride, whatever the tensor's own row shape."""
        n = self.source_rows * B.moe_row_bytes(self.H, quant)
        return self.send.view(-1)[s * n:(s + 1) * n]

    def send_scales_of(self, s: int) -> torch.Tensor:
        """Scales of source s's send rows."""
        return self.send_scales[s * self.source_rows:(s + 1) * self.source_rows]

    def _exchange(self, send, send_scales, recv, recv_scales, quant, reverse, st):
        HN.moe_exchange_blocks(send, send_scales, self.source_rows, recv, recv_scales,
                               self.max_rows, self.H, quant, self.src_offsets, self.E, self.R,
                               self.rl, reverse, st)

    @_group_device
    def run(self, logits: torch.Tensor, x: torch.Tensor, out: torch.Tensor, quant: int = 0,
            capacity_factor=None, timer: KernelTimer | None = None,
            balance: B.Balance | None = None, token_mask: torch.Tensor | None = None):
        """One layer; `balance` (alloc_balance of T tokens) also takes the
        balance loss of the tokens that token_mask keeps.  A masked token is
        routed like any other."""
        T, H, E, k, R = self.T, self.H, self.E, self.k, self.R
        if logits.shape != (T, E) or x.shape[0] != T or out.shape[0] != T:
            raise ValueError("logits/x/out shapes do not match the group")
        self._last = None  # the buffers are overwritten from here on
        st = torch.cuda.current_stream(self.device)
        M = self.max_rows
        timed = self._timed(timer, st)
        timed("route", lambda: B.moe_route_topk(logits, k, self.idx[:T], self.w[:T], st))
        if balance is not None:
            timed("balance", lambda: B.moe_balance_loss(logits, self.idx[:T], token_mask, balance,
                                                        st))
        caps = self._source_caps(capacity_factor) if capacity_factor else None
        timed("layout", lambda: B.moe_dispatch_layout_chunks(self.idx, T, E, k, R, 0, caps,
                                                              self.lay, st))
        for s, (t0, t1) in enumerate(self.bounds):
            if t1 > t0:
                timed("pack", lambda: B.moe_dispatch_pack(x[t0:t1], t1 - t0, H, k,
                                                          self.views[s].pos, quant,
                                                          self.send_rows(s, quant),
                                                          self.send_scales_of(s), st))
        so = self.src_offsets
        timed("recv_layout", lambda: B.moe_recv_layout(so, E, R, self.rl, st))
        timed("exchange", lambda: self._exchange(self.send, self.send_scales, self.recv,
                                                 self.recv_scales, quant, False, st))
        if self.experts is not None:
            self._run_experts(quant, timed, st)
        else:
            self._run_grouped(quant, timed, st)
        timed("exchange_back", lambda: self._exchange(self.send, self.send_scales, self.recv,
                                                      self.recv_scales, quant, True, st))
        for s, (t0, t1) in enumerate(self.bounds):
            if t1 > t0:
                timed("combine", lambda: B.moe_combine(
                    self.send_rows(s, quant), self.send_scales_of(s), quant, self.views[s].pos,
                    self.w[t0:t1], t1 - t0, H, k, out[t0:t1], st))
        if self.experts is not None and self.experts.train:
            self._last = (logits, quant, balance, token_mask)
            self._forward = self.experts.forwards
        return out

    @staticmethod
    def _timed(timer, st):
        def timed(name, fn):
            tok = timer.start(name, st) if timer else None
            fn()
            if timer:
                timer.stop(tok)

        return timed

    def _run_grouped(self, quant, timed, st):
        """Regroup, [stand-in] and ungroup, in the payload's format."""
        H, E, M = self.H, self.E, self.max_rows
        timed("regroup", lambda: B.moe_recv_regroup(
            self.recv, self.recv_scales, M, H, quant, self.rl.group_src, self.grouped,
            self.grouped_scales, st))
        ret, ret_scales = self.grouped, self.grouped_scales
        if self.standin:
            timed("standin", lambda: HN.moe_expert_standin(
                self.grouped, self.grouped_scales, quant, self.rl.group_offsets, E, M, H, quant,
                self.ret, self.ret_scales, st))
            ret, ret_scales = self.ret, self.ret_scales
        timed("ungroup", lambda: B.moe_recv_ungroup(ret, ret_scales, M, H, quant,
                                                    self.rl.group_pos, self.recv,
                                                    self.recv_scales, st))

    def _run_experts(self, quant, timed, st):
        """Regroup to bf16, the experts, and ungroup to the payload's format."""
        H, M, rl = self.H, self.max_rows, self.rl
        x, y = self.expert_in, self.expert_out
        if quant == B.MOE_QUANT_BF16:
            timed("regroup", lambda: B.moe_recv_regroup(self.recv, None, M, H, quant, rl.group_src,
                                                        x, None, st))
        else:
            timed("regroup", lambda: B.moe_combine(self.recv, self.recv_scales, quant,
                                                   rl.group_src, self.ones, M, H, 1, x, st))
        timed("experts", lambda: self.experts.forward(x, rl.group_offsets, y, stream=st))
        if quant == B.MOE_QUANT_BF16:
            timed("ungroup", lambda: B.moe_recv_ungroup(y, None, M, H, quant, rl.group_pos,
                                                        self.recv, None, st))
        else:
            timed("ungroup", lambda: B.moe_dispatch_pack(y, M, H, 1, rl.group_src, quant,
                                                         self.recv, self.recv_scales, st))

    @_group_device
    def backward(self, d_out: torch.Tensor, d_x: torch.Tensor | None, d_logits: torch.Tensor,
                 grads: ExpertGrads | None = None, d_loss: torch.Tensor | None = None,
                 accumulate: bool = False, timer: KernelTimer | None = None,
                 masked_gates: bool = False):
        """Gradients of the last run() from that of its output (d_out bf16
        [T, H]) and of its balance loss (d_loss fp32, one value per segment,
        or None): d_x bf16 [T, H] or None, d_logits fp32 [T, E], the experts'
        grads or None.  The run's logits, mask, Balance and this group's
        buffers must still hold what the run left in them; d_x and grads are
        refused if the experts have run for another call since.  Tokens that
        token_mask leaves out get no logit gradient, as suits padding, whose
        d_out is 0; where they only leave the balance loss and their d_out
        counts, masked_gates gives them that of their gate weights, and
        d_logits is the run's derivative for every d_out."""
        if self.experts is None or not self.experts.train:
            raise ValueError("backward needs experts with train=True")
        if self._last is None:
            raise ValueError("backward before run")
        logits, quant, balance, mask = self._last
        T, H, k, M, rl = self.T, self.H, self.k, self.max_rows, self.rl
        for t, name in ((d_out, "d_out"), (d_x, "d_x")):
            if t is not None:
                B._want_bf16(t, (T, H), name)
        if d_loss is not None and balance is None:
            raise ValueError("d_loss needs a run with a Balance")
        if (d_x is not None or grads is not None) and self._forward != self.experts.forwards:
            raise ValueError("the experts have run again since this group's run")
        st = torch.cuda.current_stream(self.device)
        timed = self._timed(timer, st)
        so = self.source_rows
        for s, (t0, t1) in enumerate(self.bounds):
            if t1 > t0:
                timed("combine_grad", lambda: B.moe_combine_grad(
                    d_out[t0:t1], self.send_rows(s, quant), self.send_scales_of(s), quant,
                    self.views[s].pos, self.w[t0:t1], t1 - t0, H, k,
                    self.d_send[s * so:(s + 1) * so], self.d_w[t0:t1], st))
        timed("route_grad", lambda: B.moe_route_grad(
            logits, self.idx[:T], self.w[:T], self.d_w[:T], mask, d_loss, balance, d_logits, st,
            masked_gates))
        if d_x is None and grads is None:
            return
        timed("exchange", lambda: self._exchange(self.d_send, None, self.d_recv, None, 0, False,
                                                 st))
        timed("regroup", lambda: B.moe_recv_regroup(self.d_recv, None, M, H, 0, rl.group_src,
                                                    self.d_rows, None, st))
        timed("experts_grad", lambda: self.experts.backward(
            self.d_rows, self.expert_in, rl.group_offsets, None if d_x is None else self.d_rows,
            grads, accumulate, st, self._forward))
        if d_x is None:
            return
        timed("ungroup", lambda: B.moe_recv_ungroup(self.d_rows, None, M, H, 0, rl.group_pos,
                                                    self.d_recv, None, st))
        timed("exchange_back", lambda: self._exchange(self.d_send, None, self.d_recv, None, 0, True,
                                                      st))
        for s, (t0, t1) in enumerate(self.bounds):
            if t1 > t0:
                timed("combine", lambda: B.moe_combine(
                    self.d_send[s * so:(s + 1) * so], None, 0, self.views[s].pos, self.ones,
                    t1 - t0, H, k, d_x[t0:t1], st))
