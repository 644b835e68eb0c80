"""Buffer plumbing around the C ABI: allocates the caller-owned device buffers with torch and
calls the entry points in order. It holds no layer arithmetic. Every step runs in the
library's kernels, and torch only provides memory and the stream.
"""
from __future__ import annotations

import torch

from . import (MOE_ACT_SILU, MOE_ERR_INVALID_ARG, MOE_FLAG_BF16_DW, MOE_FLAG_MXFP8_WGRAD,
               MOE_FLAG_PERSISTENT, MOE_PREC_BF16, MOE_PREC_INT8, MOE_PREC_MXFP4, MOE_PREC_MXFP8,
               MoeError, _dev, make_cfg, make_ffn, moe_backward, moe_ffn_backward,
               moe_ffn_forward, moe_ffn_query, moe_forward, moe_forward_fused,
               moe_gate_backward, moe_permute, moe_query, moe_quantize_weights, moe_route,
               moe_route_gated, moe_router_backward)


class SharedExpert:
    """Caller-owned buffers of the dense gated feed-forward block (``moe_ffn_forward``,
    ``moe_ffn_backward``): the expert every token passes beside its routed ones, or a block of its
    own. ``train`` keeps H = [g | u] for the backward and owns the gradients dw1 and dw2. A caller
    with several batches on their way gives each its own ``saved``, from ``new_saved``."""

    def __init__(self, T, d, I, act=MOE_ACT_SILU, device="cuda", train=True, bf16_dw=False):
        self.cfg = make_ffn(T, d, I, act, MOE_FLAG_BF16_DW if bf16_dw else 0)
        dev, bf = torch.device(device), torch.bfloat16
        self.workspace = torch.empty(moe_ffn_query(self.cfg).workspace, dtype=torch.uint8,
                                     device=dev)
        self.train = train
        self.H, self.A = self.new_saved()
        dwt = bf if bf16_dw else torch.float32
        self.dw1 = torch.zeros(2 * I, d, dtype=dwt, device=dev) if train else None
        self.dw2 = torch.zeros(d, I, dtype=dwt, device=dev) if train else None

    def new_saved(self):
        """(H, A): what one batch's forward stores for its backward."""
        T, I, bf, dev = self.cfg.T, self.cfg.I, torch.bfloat16, self.workspace.device
        return (torch.empty(T, 2 * I, dtype=bf, device=dev) if self.train else None,
                torch.empty(T, I, dtype=bf, device=dev))

    def forward(self, x, w1, w2, y, accumulate=False, stream=None, saved=None):
        """y = block(x), or with ``accumulate`` y + block(x)."""
        H, A = (self.H, self.A) if saved is None else saved
        moe_ffn_forward(self.cfg, x, w1, w2, H, A, y, accumulate, self.workspace, stream)

    def backward(self, x, w1, w2, dy, dx, accumulate_dx=False, accumulate=False, stream=None,
                 saved=None):
        """dx (added to with ``accumulate_dx``), dw1 and dw2 (added to with ``accumulate``)."""
        H, A = (self.H, self.A) if saved is None else saved
        if H is None:
            raise ValueError("a block made without train keeps nothing for a backward")
        moe_ffn_backward(self.cfg, x, w1, w2, H, A, dy, dx, self.dw1, self.dw2, accumulate_dx,
                         accumulate, self.workspace, stream)


class MoeLayer:
    """Caller-owned buffers for one (T, d, E, k, I) shape on one device.

    ``ring_slots`` slots of T*k permuted rows make up the ring. Forward writes slot ``slot``,
    and backward reads the slot its batch was permuted into. With ``precision=MOE_PREC_MXFP8``
    or ``MOE_PREC_MXFP4`` the layer also owns the quantised-weight buffer ``wq``;
    ``quantize_weights`` fills it, and ``mx_wgrad`` (MXFP8 only) makes the weight gradients
    MXFP8 too. ``MOE_PREC_FP8`` owns and fills ``wq`` likewise; its ring slots hold bf16 tokens.
    ``bf16_dw`` keeps dw1 and dw2 in bf16. ``MOE_PREC_INT8`` owns and fills ``wq`` too, and is for
    inference: it has no gradients, and no H, and its forward takes None for w1 and w2.

    With ``shared`` (a ``SharedExpert`` of the same T and d) the forward adds the shared expert's
    output to y and the backward its gradient to dx; both then need the tokens ``x`` and its weights
    ``shared_w`` = (w1, w2), and a batch with a ``saved`` of its own also a ``shared_saved``
    (``SharedExpert.new_saved``).

    With ``gate`` (from ``make_gate``) the layer routes by that gate instead of the renormalised
    top-k softmax, with ``gate_bias`` (fp32 [E], or None) in its choice, and backward takes the
    router's gradients through it; ``dlogits`` holds the logits' gradient. The single-launch
    forward has no gate, and refuses one.
    """

    def __init__(self, T, d, E, k, I, device="cuda", ring_slots=1, persistent=False,
                 precision=MOE_PREC_BF16, mx_wgrad=False, bf16_dw=False, gate=None, gate_bias=None,
                 shared=None):
        self.T, self.d, self.E, self.k, self.I = T, d, E, k, I
        flags = ((MOE_FLAG_PERSISTENT if persistent else 0) |
                 (MOE_FLAG_MXFP8_WGRAD if mx_wgrad else 0) | (MOE_FLAG_BF16_DW if bf16_dw else 0))
        self.cfg = make_cfg(T, d, E, k, I, precision, flags)
        s = moe_query(self.cfg)
        self.sizes = s
        dev = torch.device(device)
        u8, i32, f32, bf = torch.uint8, torch.int32, torch.float32, torch.bfloat16
        Tk = T * k
        self.ring = torch.empty(s.ring_slot * ring_slots, dtype=u8, device=dev)
        self.workspace = torch.empty(s.workspace, dtype=u8, device=dev)
        self.saved = torch.empty(s.saved, dtype=u8, device=dev)
        self.logits = torch.empty(T, E, dtype=f32, device=dev)
        self.topk_idx = torch.empty(T, k, dtype=i32, device=dev)
        self.topk_w = torch.empty(T, k, dtype=f32, device=dev)
        self.counts = torch.empty(E, dtype=i32, device=dev)
        self.offsets = torch.empty(E + 1, dtype=i32, device=dev)
        self.row_src = torch.empty(Tk, dtype=i32, device=dev)
        self.tk_row = torch.empty(Tk, dtype=i32, device=dev)
        self.y = torch.empty(T, d, dtype=bf, device=dev)
        self.dx = torch.empty(T, d, dtype=bf, device=dev)
        self.d_topk_w = torch.empty(T, k, dtype=f32, device=dev)
        dwt = bf if bf16_dw else f32
        self.infer = precision == MOE_PREC_INT8
        self.dw1 = None if self.infer else torch.zeros(E, 2 * I, d, dtype=dwt, device=dev)
        self.dw2 = None if self.infer else torch.zeros(E, d, I, dtype=dwt, device=dev)
        self.dwr = None if self.infer else torch.zeros(E, d, dtype=f32, device=dev)
        if shared is not None and (shared.cfg.T, shared.cfg.d) != (T, d):
            raise ValueError("the shared expert takes other tokens than the layer")
        self.shared = shared
        self.mx = precision in (MOE_PREC_MXFP8, MOE_PREC_MXFP4)
        self.fbits = 8 if precision == MOE_PREC_MXFP8 else 4 if precision == MOE_PREC_MXFP4 else 16
        self.wq = torch.empty(s.wq, dtype=u8, device=dev) if s.wq else None
        self.gate, self.gate_bias = gate, gate_bias
        self.given = False  # whether topk_idx came from set_routing, without logits
        self.dlogits = torch.empty(T, E, dtype=f32, device=dev) if gate is not None else None

    # views of intermediates -----------------------------------------------------------------
    def _view(self, buf, off, rows, cols):
        n = rows * cols * 2
        return buf[off:off + n].view(torch.bfloat16).view(rows, cols)

    def xp(self, slot=0):
        """The slot's bf16 Xp (BF16 mode), or (codes, scale codes [T*k, d/32]) as uint8 tensors:
        E4M3 codes [T*k, d] (MXFP8 mode) or E2M1 codes two a byte [T*k, d/2], element 2i in the
        low nibble (MXFP4 mode)."""
        base = slot * self.sizes.ring_slot
        if not self.mx:
            return self._view(self.ring, base, self.T * self.k, self.d)
        Tk, d = self.T * self.k, self.d
        nb = d * self.fbits // 8
        codes = self.ring[base:base + Tk * nb].view(Tk, nb)
        sc0 = base + (Tk * nb + 255) // 256 * 256
        return codes, self.ring[sc0:sc0 + Tk * d // 32].view(Tk, d // 32)

    def H(self):
        if self.infer:
            raise ValueError("the INT8 mode keeps no H")
        return self._view(self.saved, self.sizes.saved_H, self.T * self.k, 2 * self.I)

    def A(self):
        return self._view(self.saved, self.sizes.saved_A, self.T * self.k, self.I)

    def O(self):
        return self._view(self.workspace, self.sizes.ws_O, self.T * self.k, self.d)

    def dH(self):
        return self._view(self.workspace, self.sizes.ws_dH, self.T * self.k, 2 * self.I)

    def dXp(self):
        return self._view(self.workspace, self.sizes.ws_dXp, self.T * self.k, self.d)

    def device_status(self):
        return int(self.workspace[:4].view(torch.int32).item())

    # steps ----------------------------------------------------------------------------------
    def route(self, x, w_router, stream=None):
        self.given = False
        if self.gate is not None:
            moe_route_gated(self.cfg, self.gate, x, w_router, self.gate_bias, self.logits,
                            self.topk_idx, self.topk_w, self.workspace, stream)
            return
        moe_route(self.cfg, x, w_router, self.logits, self.topk_idx, self.topk_w, self.workspace,
                  stream)

    def set_routing(self, topk_idx, topk_w):
        self.given = True
        self.topk_idx.copy_(topk_idx)
        self.topk_w.copy_(topk_w)

    def permute(self, x, slot=0, stream=None):
        moe_permute(self.cfg, self.topk_idx, x, self.ring, slot, self.counts, self.offsets,
                    self.row_src, self.tk_row, self.workspace, stream)

    def quantize_weights(self, w1, w2, stream=None):
        moe_quantize_weights(self.cfg, w1, w2, self.wq, stream)

    def _shared_operands(self, x, shared_w, saved, shared_saved):
        if x is None or shared_w is None or any(w is None for w in shared_w):
            raise ValueError("a layer with a shared expert needs x and shared_w")
        if (saved is None) != (shared_saved is None):
            raise ValueError("a batch's saved and shared_saved are given together")
        return x, *shared_w

    def forward(self, w1, w2, slot=0, saved=None, stream=None, x=None, shared_w=None,
                shared_saved=None):
        """A shared expert's x, weights or buffers that ``moe_ffn_forward`` refuses are refused behind
        the routed experts' forward: y then holds their output alone until a call that goes through."""
        if self.shared is not None:
            ops = self._shared_operands(x, shared_w, saved, shared_saved)
        moe_forward(self.cfg, self.ring, slot, self.offsets, self.tk_row, self.topk_w, w1, w2,
                    self.wq, self.y, self.saved if saved is None else saved, self.workspace,
                    stream)
        if self.shared is not None:
            self.shared.forward(*ops, self.y, True, stream, shared_saved)

    def forward_fused(self, x, w_router, w1, w2, slot=0, saved=None, stream=None, shared_w=None,
                      shared_saved=None):
        """route + permute + forward in one kernel launch (moe_forward_fused), which has no gate."""
        if self.gate is not None:
            raise ValueError("the single-launch forward routes by the top-k softmax only")
        if self.shared is not None:
            ops = self._shared_operands(x, shared_w, saved, shared_saved)
        self.given = False
        moe_forward_fused(self.cfg, x, w_router, self.logits, self.topk_idx, self.topk_w,
                          self.ring, slot, self.counts, self.offsets, self.row_src, self.tk_row,
                          w1, w2, self.y, self.saved if saved is None else saved, self.workspace,
                          stream)
        if self.shared is not None:
            self.shared.forward(*ops, self.y, True, stream, shared_saved)

    def _trains(self):
        if self.infer:
            raise ValueError("the INT8 mode has no backward")

    # What a call behind moe_backward would refuse is refused before the experts' gradients are
    # written or added to: a corrected call would add a batch's a second time.
    def _before_gradients(self, stream, *args):
        _dev("MoeLayer.backward", stream, *args)
        if any(t is not None and t.data_ptr() % 16 for t, _, _ in args):
            raise MoeError(MOE_ERR_INVALID_ARG, "MoeLayer.backward: a tensor that starts at a "
                           "multiple of 16 bytes expected")

    def _not_dx(self, *args):
        if any(t is not None and t.data_ptr() == self.dx.data_ptr() for t in args):
            raise MoeError(MOE_ERR_INVALID_ARG, "MoeLayer.backward: dx is neither x nor dy")

    def backward(self, w_router, w1, w2, dy, slot=0, accumulate=False, saved=None, stream=None,
                 x=None, shared_w=None, shared_saved=None):
        """With a gate and a ``w_router``, ``x`` (the tokens) is needed too: the experts' backward
        runs as for a given routing, then the gate's and the router's add theirs to dx and dwr.
        With a shared expert its backward comes last and adds to dx."""
        self._trains()
        T, d, bf = self.T, self.d, torch.bfloat16
        if self.shared is not None:
            ops = self._shared_operands(x, shared_w, saved, shared_saved)
            sh, I = self.shared, self.shared.cfg.I
            H, A = (sh.H, sh.A) if shared_saved is None else shared_saved
            if sh.H is None or H is None or A is None:
                raise ValueError("the shared expert was made without train, or the batch's saved was")
            dw = bf if sh.cfg.flags & MOE_FLAG_BF16_DW else torch.float32
            self._before_gradients(stream, (x, bf, T * d), (ops[1], bf, 2 * I * d),
                                   (ops[2], bf, d * I), (dy, bf, T * d), (H, bf, T * 2 * I),
                                   (A, bf, T * I), (sh.dw1, dw, 2 * I * d), (sh.dw2, dw, d * I),
                                   (sh.workspace, torch.uint8, 0), (self.dx, bf, T * d))
            self._not_dx(x, dy)
        gated = self.gate is not None and w_router is not None
        if gated:
            if self.given:
                raise ValueError("a given routing has no logits to take a gate's gradients at")
            if x is None:
                raise ValueError("a gated layer's router gradients need x")
            self._before_gradients(stream, (x, bf, T * d), (w_router, bf, self.E * d))
            self._not_dx(x)
        routed = w_router is not None and not gated
        moe_backward(self.cfg, self.ring, slot, self.offsets, self.row_src, self.tk_row,
                     self.topk_idx, self.topk_w, w_router if routed else None, w1, w2, self.wq,
                     self.saved if saved is None else saved, dy, self.dx, self.dw1, self.dw2,
                     self.dwr if routed else None, self.d_topk_w, accumulate,
                     self.workspace, stream)
        if gated:
            moe_gate_backward(self.cfg, self.gate, self.logits, self.topk_idx, self.d_topk_w,
                              self.dlogits, False, stream)
            moe_router_backward(self.cfg, x, w_router, self.dlogits, self.dx, self.dwr, True,
                                accumulate, stream)
        if self.shared is not None:
            self.shared.backward(*ops, dy, self.dx, True, accumulate, stream, shared_saved)

    def step(self, x, w_router, w1, w2, dy, slot=0, stream=None, fused=False, shared_w=None):
        """One fwd+bwd pass: route (when w_router is given), permute, forward, backward. With
        ``fused`` the first three run as one launch (moe_forward_fused)."""
        self._trains()  # before anything runs
        if self.shared is not None:
            self._shared_operands(x, shared_w, None, None)
            if self.shared.H is None:
                raise ValueError("the shared expert was made without train")
        if fused:
            self.forward_fused(x, w_router, w1, w2, slot, stream=stream, shared_w=shared_w)
            self.backward(w_router, w1, w2, dy, slot, stream=stream, x=x, shared_w=shared_w)
            return
        if w_router is not None:
            self.route(x, w_router, stream)
        self.permute(x, slot, stream)
        self.forward(w1, w2, slot, stream=stream, x=x, shared_w=shared_w)
        self.backward(w_router, w1, w2, dy, slot, stream=stream, x=x, shared_w=shared_w)


class Macrobatch:
    """The streaming macrobatch: ``n`` microbatches through one fixed ring of ``ring_bytes``.

    Forward runs microbatches 0..n-1, microbatch i in slot i mod S with S = ring slots that fit;
    backward walks n-1..0 and re-permutes (replays) a microbatch whose slot a later one
    overwrote, accumulating the weight gradients in that fixed order (MarkTechPost, "Three
    design decisions that matter": the ring is walked in reverse in backward). Each microbatch
    keeps its own routing, saved activations and outputs.

    With ``overlap`` the router and permutation of the next microbatch (and, in backward, the
    replay of the next one down) run on a second stream while the current microbatch's grouped
    GEMMs run on the first, with their own workspace; events order the two. Every kernel still
    sees exactly the same inputs, so results are bitwise those of the serial walk.
    """

    def __init__(self, T, d, E, k, I, n, ring_bytes, device="cuda", overlap=False, fused=False):
        self.T, self.d, self.E, self.k, self.I, self.n = T, d, E, k, I, n
        self.main = MoeLayer(T, d, E, k, I, device=device, ring_slots=1)
        s = self.main.sizes
        self.S = ring_bytes // s.ring_slot
        if self.S < 1:
            raise ValueError("ring_bytes holds no ring slot")
        self.main.ring = torch.empty(self.S * s.ring_slot, dtype=torch.uint8, device=device)
        self.overlap = overlap
        self.fused = fused  # each microbatch's route + permute + forward as one launch
        dev = torch.device(device)
        i32, f32, bf = torch.int32, torch.float32, torch.bfloat16
        Tk = T * k
        self.route_ws = torch.empty(s.workspace, dtype=torch.uint8, device=dev) if overlap else None
        self.side = torch.cuda.Stream(device=dev) if overlap else None
        self.mb = []
        for _ in range(n):
            self.mb.append(dict(
                logits=torch.empty(T, E, dtype=f32, device=dev),
                topk_idx=torch.empty(T, k, dtype=i32, device=dev),
                topk_w=torch.empty(T, k, dtype=f32, device=dev),
                counts=torch.empty(E, dtype=i32, device=dev),
                offsets=torch.empty(E + 1, dtype=i32, device=dev),
                row_src=torch.empty(Tk, dtype=i32, device=dev),
                tk_row=torch.empty(Tk, dtype=i32, device=dev),
                saved=torch.empty(s.saved, dtype=torch.uint8, device=dev),
                y=torch.empty(T, d, dtype=bf, device=dev),
                dx=torch.empty(T, d, dtype=bf, device=dev),
                d_topk_w=torch.empty(T, k, dtype=f32, device=dev)))

    @property
    def dw1(self):
        return self.main.dw1

    @property
    def dw2(self):
        return self.main.dw2

    @property
    def dwr(self):
        return self.main.dwr

    def _route_permute(self, i, x, w_router, ws, stream, route=True):
        b, L = self.mb[i], self.main
        if route:
            moe_route(L.cfg, x, w_router, b["logits"], b["topk_idx"], b["topk_w"], ws, stream)
        moe_permute(L.cfg, b["topk_idx"], x, L.ring, i % self.S, b["counts"], b["offsets"],
                    b["row_src"], b["tk_row"], ws, stream)

    def _forward(self, i, w1, w2, stream):
        b, L = self.mb[i], self.main
        moe_forward(L.cfg, L.ring, i % self.S, b["offsets"], b["tk_row"], b["topk_w"], w1, w2,
                    None, b["y"], b["saved"], L.workspace, stream)

    def _backward(self, i, w_router, w1, w2, dy, stream):
        b, L = self.mb[i], self.main
        moe_backward(L.cfg, L.ring, i % self.S, b["offsets"], b["row_src"], b["tk_row"],
                     b["topk_idx"], b["topk_w"], w_router, w1, w2, None, b["saved"], dy, b["dx"],
                     L.dw1, L.dw2, L.dwr, b["d_topk_w"], int(i != self.n - 1), L.workspace,
                     stream)

    def run(self, X, w_router, w1, w2, dY, stream=None):
        """X and dY: [n, T, d] bf16. One macrobatch: forward 0..n-1, backward n-1..0."""
        main = torch.cuda.current_stream() if stream is None else stream
        n, S = self.n, self.S
        replay = lambda i: i < n - S  # its slot was overwritten by microbatch i + S
        if self.fused:
            for i in range(n):
                b, L = self.mb[i], self.main
                moe_forward_fused(L.cfg, X[i], w_router, b["logits"], b["topk_idx"],
                                  b["topk_w"], L.ring, i % S, b["counts"], b["offsets"],
                                  b["row_src"], b["tk_row"], w1, w2, b["y"], b["saved"],
                                  L.workspace, main)
            for i in reversed(range(n)):
                if replay(i):
                    self._route_permute(i, X[i], w_router, self.main.workspace, main, False)
                self._backward(i, w_router, w1, w2, dY[i], main)
            return
        if not self.overlap or S < 2:  # one slot: each microbatch waits for the previous one
            for i in range(n):
                self._route_permute(i, X[i], w_router, self.main.workspace, main)
                self._forward(i, w1, w2, main)
            for i in reversed(range(n)):
                if replay(i):
                    self._route_permute(i, X[i], w_router, self.main.workspace, main, False)
                self._backward(i, w_router, w1, w2, dY[i], main)
            return
        side = self.side
        ready = [torch.cuda.Event() for _ in range(n)]   # microbatch i routed and permuted
        slot_free = [torch.cuda.Event() for _ in range(n)]  # microbatch i done with its slot
        side.wait_stream(main)
        self._route_permute(0, X[0], w_router, self.route_ws, side)
        ready[0].record(side)
        for i in range(n):
            if i + 1 < n:
                if i + 1 >= S:  # slot (i+1) mod S last held microbatch i+1-S
                    side.wait_event(slot_free[i + 1 - S])
                self._route_permute(i + 1, X[i + 1], w_router, self.route_ws, side)
                ready[i + 1].record(side)
            main.wait_event(ready[i])
            self._forward(i, w1, w2, main)
            slot_free[i].record(main)
        # backward: the replay of microbatch i-1 overlaps the backward of microbatch i
        done = [torch.cuda.Event() for _ in range(n)]  # backward of microbatch i finished
        for i in reversed(range(n)):
            j = i - 1
            if j >= 0 and replay(j):
                # slot j mod S holds microbatch j+S (> i, walked already): its backward must be
                # done with the slot before the replay overwrites it
                side.wait_event(done[j + S])
                self._route_permute(j, X[j], w_router, self.route_ws, side, False)
                ready[j].record(side)
            if replay(i):
                main.wait_event(ready[i])
            self._backward(i, w_router, w1, w2, dY[i], main)
            done[i].record(main)
        main.wait_stream(side)
