"""Device-resident MoE layers, and the expert order for training.

Memory management and marshalling only (torch allocates, the library
computes).  W4A16MoELayer uploads its weights once, repacked on the device by
chord_w4a16_prepack; forward() is one chord_moe_layer call.  MXFP4MoELayer
keeps MXFP4 weights and runs the experts with both operands in 4 bits.
ExpertOrder holds a routing's aligned expert order, and permute_rows /
unpermute_rows move rows into it and back with gradients.  expert_product and
expert_mlp train the experts in 16 bits between the two, expert_mlp with the
activations that its backward pass needs held in 8.
"""
from __future__ import annotations

import contextlib

import numpy as np
import torch
from torch.autograd.function import once_differentiable

from . import chord


def to_device(a, device="cuda"):
    """numpy array -> torch tensor on device (uint16 arrays become bfloat16)."""
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        return torch.from_numpy(a.view(np.int16)).to(device).view(torch.bfloat16)
    return torch.from_numpy(a).to(device)


def _on_stream(stream):
    """A context in which torch allocates and copies on `stream` (a stream, a raw handle, or
    None: the current one), and calls without a stream run: memory that it frees there is
    handed out again behind that stream's work only."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(getattr(stream, "cuda_stream", stream))
    return torch.cuda.stream(stream)


def prepack(q, s, gate_up: bool, stream=None):
    """Device uint8 [E,N,K/2] + bfloat16 [E,N,K/32] -> packed blob (uint8 tensor)."""
    E, N, K2 = q.shape
    nbytes = chord.chord_w4a16_prepack_bytes(E, N, 2 * K2)
    packed = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    chord.chord_w4a16_prepack(q, s, gate_up, packed, stream=stream)
    return packed


class W4A16MoELayer:
    """One expert shard of a MoE layer (local experts [expert_begin, +E_local))."""

    def __init__(self, w13_q, w13_s, w2_q, w2_s, E_total: int, expert_begin: int, topk: int,
                 device="cuda"):
        w13_q, w13_s = to_device(w13_q, device), to_device(w13_s, device)
        w2_q, w2_s = to_device(w2_q, device), to_device(w2_s, device)
        self.E_local, twoI, H2 = w13_q.shape
        self.H, self.I = 2 * H2, twoI // 2
        self.E_total, self.expert_begin, self.topk = E_total, expert_begin, topk
        self.w13 = prepack(w13_q, w13_s, True)
        self.w2 = prepack(w2_q, w2_s, False)
        torch.cuda.synchronize()
        self._ws = None
        self._ws_M = -1
        self.dev_status = torch.zeros(1, dtype=torch.int32, device=device)

    def workspace(self, M: int):
        if M > self._ws_M:
            n = chord.chord_moe_layer_workspace_bytes(M, self.H, self.I, self.E_local, self.topk)
            self._ws = torch.empty(max(n, 1), dtype=torch.uint8, device=self.w13.device)
            self._ws_M = M
        return self._ws

    def forward(self, x, logits, bias, out=None, topk_weights_out=None, topk_ids_out=None,
                tuning=None, stream=None):
        M = x.shape[0]
        if out is None:
            out = torch.empty((M, self.H), dtype=torch.bfloat16, device=x.device)
        chord.chord_moe_layer(x, logits, bias, self.w13, self.w2, self.H, self.I, self.E_total,
                              self.expert_begin, self.E_local, self.topk, out, self.workspace(M),
                              topk_weights_out, topk_ids_out, tuning=tuning,
                              dev_status=self.dev_status, stream=stream)
        return out


class ExpertOrder:
    """The aligned order of the assignments of M tokens to topk of E_total experts, on
    one shard (local experts [expert_begin, +E_local)); route() fills it, and may fill it
    anew once the gradients of what used it have been taken (before that, they raise).

    topk_weights [M, topk] FP32 and topk_ids [M, topk]; sorted_token_ids [capacity],
    sorted_positions [M * topk], num_tokens_post_padded [1], expert_counts [E_local]
    and expert_offsets [E_local + 1], as chord_moe_align defines them; dev_status [1], for
    errors that the experts' products find on the device."""

    def __init__(self, M: int, topk: int, expert_begin: int, E_local: int, block_m: int = 16, device="cuda"):
        self.M, self.topk, self.expert_begin, self.E_local, self.block_m = M, topk, expert_begin, E_local, block_m
        self.capacity = chord.chord_moe_align_capacity(M, topk, E_local, block_m)
        i32 = dict(dtype=torch.int32, device=device)
        self.topk_weights = torch.empty((M, topk), dtype=torch.float32, device=device)
        self.topk_ids = torch.empty((M, topk), **i32)
        self.sorted_token_ids = torch.empty(self.capacity, **i32)
        self.sorted_positions = torch.empty(M * topk, **i32)
        self.expert_ids = torch.empty(self.capacity // block_m, **i32)
        self.num_tokens_post_padded = torch.empty(1, **i32)
        self.expert_counts = torch.empty(E_local, **i32)
        self.expert_offsets = torch.empty(E_local + 1, **i32)
        self.dev_status = torch.zeros(1, **i32)
        nbytes = chord.chord_moe_align_workspace_bytes(M, topk, E_local)
        self._ws = torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None
        self._arrays = (self.topk_weights, self.topk_ids, self.sorted_token_ids, self.sorted_positions,
                        self.expert_ids, self.num_tokens_post_padded, self.expert_counts, self.expert_offsets)
        # tensors made in inference mode have no versions, and cannot be saved outside it
        self._versioned = () if self.topk_weights.is_inference() else self._arrays
        self._streams = {None}   # streams that its memory may be in use on

    def _saved(self, *arrays):
        """Arrays of the order as a backward pass can keep them."""
        if self._versioned or torch.is_inference_mode_enabled():
            return arrays
        return [t.clone() for t in arrays]

    def route(self, logits, bias, stream=None):
        """Top-k routing of logits [M, E_total] and the order, on the device.  The order's memory
        is of the stream that was current when it was made: a call on another `stream` follows
        that one's work, and with a raw handle the order is kept until the call has run."""
        if logits.dim() != 2 or logits.shape[0] != self.M:
            raise ValueError(f"logits must be [{self.M}, E_total] for this order, got {list(logits.shape)}")
        if stream not in self._streams and isinstance(stream, torch.cuda.Stream):
            for t in (*self._arrays, self.dev_status, *([] if self._ws is None else [self._ws])):
                t.record_stream(stream)
            self._streams.add(stream)
        if self.M == 0:   # arrays without elements have no address to give
            with _on_stream(stream):
                for t in (self.num_tokens_post_padded, self.expert_counts, self.expert_offsets):
                    t.zero_()
            return self
        chord.chord_moe_route_align(logits, bias, self.topk, self.expert_begin, self.E_local, self.block_m,
                                    self.topk_weights, self.topk_ids, self.sorted_token_ids, self.expert_ids,
                                    self.num_tokens_post_padded, self.expert_counts, self.expert_offsets,
                                    self.sorted_positions, self._ws, stream=stream)
        # written through raw pointers: autograd is told, as of any write in place
        torch.autograd.graph.increment_version(self._versioned)
        return self


def _unit_columns(g):
    """A gradient as rows with unit column stride (that of a sum has stride 0 everywhere)."""
    return g if g.stride(1) == 1 or g.shape[1] == 1 else g.contiguous()


def _once(backward):
    """once_differentiable, but only where a graph of the gradient is asked for: its wrapping
    takes the host 2 us a call."""
    checked = once_differentiable(backward)
    return lambda ctx, *grads: (checked if torch.is_grad_enabled() else backward)(ctx, *grads)


# The maps are saved like any tensor, so that a backward after route() has filled the order
# anew is an error instead of the gradient of another routing.
class _Permute(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, order):
        ctx.M, ctx.topk = order.M, order.topk
        ctx.save_for_backward(*order._saved(order.sorted_positions))
        # rows past the padded total are not written by the call: zeros
        out = torch.zeros((order.capacity, x.shape[1]), dtype=x.dtype, device=x.device)
        chord.chord_moe_permute(x, order.sorted_positions, order.sorted_token_ids, order.num_tokens_post_padded,
                                order.topk, out)
        return out

    @staticmethod
    @_once
    def backward(ctx, dout):
        positions, = ctx.saved_tensors
        dout = _unit_columns(dout)
        dx = torch.empty((ctx.M, dout.shape[1]), dtype=dout.dtype, device=dout.device)
        chord.chord_moe_permute_backward(dout, positions, ctx.topk, dx)
        return dx, None


class _Unpermute(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, weights, order):
        ctx.save_for_backward(y, weights, *order._saved(order.sorted_positions, order.sorted_token_ids,
                                                       order.num_tokens_post_padded))
        out = torch.empty((order.M, y.shape[1]), dtype=y.dtype, device=y.device)
        chord.chord_moe_unpermute(y, weights, order.sorted_positions, out)
        return out

    @staticmethod
    @_once
    def backward(ctx, dout):
        y, weights, positions, token_ids, total = ctx.saved_tensors
        dout = _unit_columns(dout)
        dy, dw = torch.zeros_like(y, memory_format=torch.contiguous_format), torch.empty_like(weights)
        chord.chord_moe_unpermute_backward(dout, y, weights, positions, token_ids, total, dy, dw)
        return dy, dw, None


def permute_rows(x, order: ExpertOrder):
    """x [M, H] -> rows [order.capacity, H] in expert order, zeros elsewhere; differentiable once
    (a second derivative raises)."""
    return _Permute.apply(x, order)


def unpermute_rows(y, weights, order: ExpertOrder):
    """The weighted sum of rows y [order.capacity, H] back to tokens [M, H]; differentiable
    once in y and in weights FP32 [M, topk] (a second derivative raises)."""
    if y.shape[0] != order.capacity:
        raise ValueError(f"y must hold the {order.capacity} rows of its order, got {y.shape[0]}")
    return _Unpermute.apply(y, weights, order)


def _rows16(t):
    """Rows as the products read them: 16-byte parts, rows apart from one another."""
    t = _unit_columns(t)
    fine = t.data_ptr() % 16 == 0 and (t.shape[0] <= 1 or (t.stride(0) % 8 == 0 and t.stride(0) >= t.shape[1]))
    return t if fine else t.clone(memory_format=torch.contiguous_format)


class _Products:
    """The products of one pass over an order's experts.  Their workspace is memory of the pass
    (or of the graph that captures it), so that passes on several streams share none."""

    def __init__(self, counts, offsets, status):
        self.counts, self.offsets, self.status = counts, offsets, status
        self.ws = torch.empty(chord.chord_expert_gemm_workspace_bytes(), dtype=torch.uint8, device=counts.device)
        self.ws[:chord.CHORD_EXPERT_GEMM_COUNTER_BYTES].zero_()

    def rows(self, x, w, transpose=False, out=None):
        if out is None:
            out = torch.empty((x.shape[0], w.shape[2 if transpose else 1]), dtype=x.dtype, device=x.device)
        chord.chord_expert_gemm(x, w, self.counts, self.offsets, out, self.ws, transpose, self.status)
        return out

    def weights(self, dout, x, like):
        dw = torch.empty_like(like, memory_format=torch.contiguous_format)
        chord.chord_expert_wgrad(dout, x, self.counts, self.offsets, dw, self.ws, self.status)
        return dw


class _ExpertProduct(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, w, order):
        ctx.status = order.dev_status
        ctx.save_for_backward(rows, w, *order._saved(order.expert_counts, order.expert_offsets))
        # rows that are no expert's are not written by the call: zeros
        out = torch.zeros((order.capacity, w.shape[1]), dtype=rows.dtype, device=rows.device)
        return _Products(order.expert_counts, order.expert_offsets, order.dev_status).rows(rows, w, out=out)

    @staticmethod
    @_once
    def backward(ctx, dout):
        rows, w, counts, offsets = ctx.saved_tensors
        products, dout = _Products(counts, offsets, ctx.status), _rows16(dout)
        drows = dw = None
        if ctx.needs_input_grad[0]:
            drows = products.rows(dout, w, True, torch.zeros(rows.shape, dtype=rows.dtype, device=rows.device))
        if ctx.needs_input_grad[1]:
            dw = products.weights(dout, rows, w)
        return drows, dw, None


def expert_product(rows, w, order: ExpertOrder):
    """rows [order.capacity, K] times each expert's w [E_local, N, K] -> [order.capacity, N], zeros in rows that
    are no expert's; BF16 or FP16, differentiable once in rows and w.

    What the products find wrong on the device (counts that are no order of the rows, a wait that ran out) is recorded
    in order.dev_status; rows and gradients are then not computed, and hold zeros or anything."""
    if rows.shape[0] != order.capacity or w.shape[0] != order.E_local:
        raise ValueError(f"rows must hold the {order.capacity} rows of the order and w its {order.E_local} experts, "
                         f"got {rows.shape[0]} and {w.shape[0]}")
    return _ExpertProduct.apply(_rows16(rows), w, order)


class _ExpertMLP(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weights, w13, w2, order, held):
        o, (M, H), I, cap = order, x.shape, w2.shape[2], order.capacity
        empty = lambda *shape, dtype=x.dtype: torch.empty(shape, dtype=dtype, device=x.device)
        codes8 = lambda n, k: (empty(n, k, dtype=torch.uint8), empty(n, k // 32, dtype=torch.uint8))
        products = _Products(o.expert_counts, o.expert_offsets, o.dev_status)
        rows, h, out = empty(cap, H), empty(cap, I), empty(M, H)
        chord.chord_moe_permute(x, o.sorted_positions, o.sorted_token_ids, o.num_tokens_post_padded, o.topk, rows)
        gu = products.rows(rows, w13)
        kept = codes8(cap, 2 * I) if held else ()
        chord.chord_swiglu(gu, weights, o.sorted_token_ids, o.num_tokens_post_padded, h, *kept)
        y = products.rows(h, w2)
        chord.chord_moe_permute_backward(y, o.sorted_positions, o.topk, out)   # the sum over a token's rows
        if not held:
            kept = (gu,)
        if ctx.needs_input_grad[2]:   # (x is needed for w13's gradient alone)
            if held:
                x8 = codes8(M, H)
                chord.chord_mxfp8_quantize(x, *x8)
                kept = (*kept, *x8)
            else:
                kept = (gu, x)
        ctx.held, ctx.topk, ctx.cap, ctx.status, ctx.dtype = held, o.topk, cap, o.dev_status, x.dtype
        ctx.save_for_backward(weights, w13, w2, *o._saved(o.sorted_positions, o.sorted_token_ids,
                                                         o.num_tokens_post_padded, o.expert_counts, o.expert_offsets),
                              *kept)
        return out

    @staticmethod
    @_once
    def backward(ctx, dout):
        weights, w13, w2, positions, token_ids, total, counts, offsets, *kept = ctx.saved_tensors
        M, (twoI, H) = dout.shape[0], w13.shape[1:]
        empty = lambda *shape: torch.empty(shape, dtype=ctx.dtype, device=dout.device)
        products = _Products(counts, offsets, ctx.status)
        dy, dgu, dweights = empty(ctx.cap, H), empty(ctx.cap, twoI), torch.empty_like(weights)
        h = empty(ctx.cap, twoI // 2) if ctx.needs_input_grad[3] else None
        chord.chord_moe_permute(_unit_columns(dout), positions, token_ids, total, ctx.topk, dy)
        dh = products.rows(dy, w2, True)
        gu, codes, kept_x = (None, kept[:2], kept[2:]) if ctx.held else (kept[0], (None, None), kept[1:])
        chord.chord_swiglu_backward(dh, gu, *codes, weights, positions, token_ids, total, dgu, dweights, h)
        dx = dw13 = dw2 = None
        if ctx.needs_input_grad[3]:
            dw2 = products.weights(dy, h, w2)
        if ctx.needs_input_grad[2]:
            rows = dy   # (used up)
            if ctx.held:
                chord.chord_mxfp8_permute(*kept_x, positions, token_ids, total, ctx.topk, rows)
            else:
                chord.chord_moe_permute(*kept_x, positions, token_ids, total, ctx.topk, rows)
            dw13 = products.weights(dgu, rows, w13)
        if ctx.needs_input_grad[0]:
            dx = empty(M, H)
            chord.chord_moe_permute_backward(products.rows(dgu, w13, True), positions, ctx.topk, dx)
        return dx, dweights if ctx.needs_input_grad[1] else None, dw13, dw2, None, None


def expert_mlp(x, weights, w13, w2, order: ExpertOrder, held_in_8_bits: bool = True):
    """The order's SiLU-gated experts over tokens x [M, H], summed back with the routing weights FP32 [M, topk]:
    out[t] = sum_j weights[t, j] w2[e] (silu(gate) * up), gate and up the halves of w13[e] x[t], e the expert of
    assignment (t, j) where it is local.  w13 [E_local, 2I, H] (rows 0..I-1 gate) and w2 [E_local, H, I]; x, w13 and
    w2 BF16 or FP16, H and I multiples of 8.  Differentiable once in x, weights, w13 and w2.

    The backward pass keeps the rows of gate and up, and x where w13 needs a gradient.  By default it keeps them in 8
    bits (MXFP8; H and I multiples of 32): the gradients of the weights and of the activation then see each kept value
    v rounded by up to 2^-4 |v|, or 2^-10 of its block's scale where that is more.  A block is 32 neighbours in a row,
    its scale at most 1/224 of the largest of them, so that values below about 2^-18 of that are kept as 0.
    held_in_8_bits=False keeps them as they are.  The output is the same either way.

    Errors on the device are recorded in order.dev_status, as for expert_product: a program that can wait reads it,
    after the backward pass too, before it trusts what it got."""
    if x.shape[0] != order.M or w13.shape[0] != order.E_local or w2.shape[0] != order.E_local:
        raise ValueError(f"x must hold the order's {order.M} tokens and w13 and w2 its {order.E_local} experts, got "
                         f"{x.shape[0]}, {w13.shape[0]} and {w2.shape[0]}")
    if w13.shape[1] != 2 * w2.shape[2] or w13.shape[2] != x.shape[1] or w2.shape[1] != x.shape[1]:
        raise ValueError(f"w13 {list(w13.shape)} and w2 {list(w2.shape)} must be [E, 2I, {x.shape[1]}] and "
                         f"[E, {x.shape[1]}, I]")
    if weights.shape != (order.M, order.topk):
        raise ValueError(f"weights must be [{order.M}, {order.topk}], got {list(weights.shape)}")
    if held_in_8_bits and (x.shape[1] % 32 or w2.shape[2] % 32):
        raise ValueError(f"H={x.shape[1]} and I={w2.shape[2]} must be multiples of 32 to be held in 8 bits")
    # nothing is kept, and nothing quantised, where no gradient can follow
    held = held_in_8_bits and torch.is_grad_enabled() and any(t.requires_grad for t in (x, weights, w13, w2))
    return _ExpertMLP.apply(_unit_columns(x), weights.contiguous(), w13, w2, order, held)


def quantize_mxfp4(w, stream=None):
    """[..., K] BF16, FP16 or FP32 on the device -> MXFP4 codes uint8 [..., K/2] and scales uint8 [..., K/32],
    made on the call's stream."""
    K = w.shape[-1]
    with _on_stream(stream):
        codes = torch.empty((*w.shape[:-1], K // 2), dtype=torch.uint8, device=w.device)
        scales = torch.empty((*w.shape[:-1], K // 32), dtype=torch.uint8, device=w.device)
        chord.chord_mxfp4_quantize(w.reshape(-1, K), codes, scales)
    return codes, scales


class MXFP4MoELayer:
    """One expert shard of a MoE layer whose experts run in MXFP4 on both operands:
    route and align, rows quantised into expert order, gate/up product with SiLU * up,
    rows quantised again, down product, weighted sum back to tokens.

    w13: (codes [E_local, 2I, H/2], scales [E_local, 2I, H/32]), rows 0..I-1 gate and
    I..2I-1 up; w2: (codes [E_local, H, I/2], scales [E_local, H, I/32]), as
    quantize_mxfp4 gives them, on the device.  Calls share the product's workspace, so they
    follow one another; each one's buffers are memory of its own stream.  Calls may be
    captured in CUDA graphs, one per batch size: the buffers of a captured call are kept
    with the layer, which has to outlive the graph."""

    def __init__(self, w13, w2, E_total: int, expert_begin: int, topk: int):
        (q13, s13), (q2, s2) = w13, w2
        self.device = q13.device
        self.E_local, twoI, self.H, self.I = q13.shape[0], q13.shape[1], 2 * q13.shape[2], 2 * q2.shape[2]
        if twoI != 2 * self.I or q2.shape[:2] != (self.E_local, self.H):
            raise ValueError("w13 must be [E_local, 2I, H/2] and w2 [E_local, H, I/2]")
        self.E_total, self.expert_begin, self.topk = E_total, expert_begin, topk
        self.w13 = self._prepack(q13, s13, True)
        self.w2 = self._prepack(q2, s2, False)
        self._ws = torch.zeros(chord.chord_mxfp4_moe_gemm_workspace_bytes(), dtype=torch.uint8, device=self.device)
        self.dev_status = torch.zeros(1, dtype=torch.int32, device=self.device)
        torch.cuda.current_stream(self.device).synchronize()   # the first call may be on any stream
        self._key = None      # (tokens, stream) of the buffers
        self._captured = {}   # buffers that captured graphs use, by (tokens, stream)

    def _prepack(self, codes, scales, gate_up):
        E, N, K2 = codes.shape
        packed = torch.empty(chord.chord_mxfp4_prepack_bytes(E, N, 2 * K2), dtype=torch.uint8, device=self.device)
        chord.chord_mxfp4_prepack(codes, scales, gate_up, packed)
        return packed

    def _allocate(self, M: int):
        """(order, row operand, h, y) for M tokens, in the current stream's memory."""
        order = ExpertOrder(M, self.topk, self.expert_begin, self.E_local, device=self.device)
        cap, bf16 = order.capacity, dict(dtype=torch.bfloat16, device=self.device)
        rows = torch.empty(max(chord.chord_mxfp4_rows_bytes(cap, self.H), chord.chord_mxfp4_rows_bytes(cap, self.I)),
                           dtype=torch.uint8, device=self.device)
        return order, rows, torch.empty((cap, self.I), **bf16), torch.empty((cap, self.H), **bf16)

    def _buffers(self, M: int):
        # of one stream only: what is dropped here may still be in use on its own
        key = (M, chord._stream(None))
        if torch.cuda.is_current_stream_capturing():
            # a graph's replays use them as long as it lives: kept, and for captures only
            if key not in self._captured:
                self._captured[key] = self._allocate(M)
            self.order, self._rows, self.h, self.y = self._captured[key]
            self._key = None
        elif key != self._key:
            self.order, self._rows, self.h, self.y = self._allocate(M)
            self._key = key
        return self.order

    def forward(self, x, logits, bias, out=None, stream=None):
        """x [M, H] (BF16, FP16 or FP32), logits FP32 [M, E_total], bias FP32 [E_total] -> out [M, H] BF16.
        A missing `out` is made on the call's stream."""
        M = x.shape[0]
        for name, t, shape in (("x", x, (M, self.H)), ("logits", logits, (M, self.E_total)),
                               ("bias", bias, (self.E_total,))):
            if t.shape != shape:
                raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
        with _on_stream(stream):
            if out is None:
                out = torch.empty((M, self.H), dtype=torch.bfloat16, device=self.device)
            if M > 0:
                self._run(x, logits, bias, out)
        return out

    def _run(self, x, logits, bias, out):
        o = self._buffers(x.shape[0]).route(logits, bias)
        cap, n = o.capacity, o.num_tokens_post_padded
        chord.chord_mxfp4_quantize_rows(x, o.sorted_positions, self.topk, n, cap, self._rows)
        chord.chord_mxfp4_moe_gemm(self._rows, self.w13, self.E_local, 2 * self.I, self.H, o.expert_counts,
                                   o.expert_offsets, cap, chord.CHORD_EPI_SILU_MUL, self.h, self._ws, self.dev_status)
        chord.chord_mxfp4_quantize_rows(self.h, None, 1, n, cap, self._rows)
        chord.chord_mxfp4_moe_gemm(self._rows, self.w2, self.E_local, self.H, self.I, o.expert_counts,
                                   o.expert_offsets, cap, chord.CHORD_EPI_STORE, self.y, self._ws, self.dev_status)
        chord.chord_moe_unpermute(self.y, o.topk_weights, o.sorted_positions, out)
