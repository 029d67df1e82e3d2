"""The routed SwiGLU layer with experts stored in 8-bit integers.

One call runs, on the current stream and without a host synchronisation:

1. the residual addition and the RMSNorm's int8 rows with a scale each:
   ``ace_add_rmsnorm``;
2. the router's logits from the sums, at fp32 accuracy: ``ace_moe_logits``;
3. experts, weights and the ACE skip mask: ``ace_gate_topk``;
4. the kept slots in expert order: ``ace_moe_group``;
5. gate and up projections of the kept slots, their rows read through the
   slots' tokens: ``ace_matmul_i8``;
6. SiLU(gate) * up, to int8 rows: ``ace_swiglu``;
7. the down projection, scaled by the slots' weights: ``ace_matmul_i8``;
8. the sum of each token's slots in rank order: ``ace_moe_combine``.

The number of kept slots stays on the device: buffers have room for every slot,
and the kernels stop at the last one in use.  The buffers are allocated once
(``LayerI8(..., max_tokens)``), so a call can be captured in a CUDA graph.  Calls of
one object share them: a call waits on the device for the one before it, whichever
stream and thread that came from.  A captured call runs when its graph is replayed;
the program orders a replay with other replays and calls of the same object.
Arithmetic is the operators' (see include/ace.h): integer sums are exact, int8
rows are correctly rounded, everything else is fp32 with one rounding per stored
result.
"""
import threading

import torch

from . import ace


def quantise_rows(w):
    """int8 rows of w [..., n] and their fp32 scales [...]: q = nearest
    integer of 127 w / max |w| of its row, scale = max |w| / 127 (0 for a row of
    zeros).  Used once per checkpoint, to store weights in 8 bits."""
    top = w.double().abs().amax(-1, keepdim=True)
    q = torch.where(top > 0, torch.round(w.double() * 127.0 / top), 0.0)
    return q.to(torch.int8), (top[..., 0] / 127.0).float()


class LayerI8:
    """Weights and buffers of one layer.

    gamma [d] fp32; w_router [E][d] in the activations' type (bf16 or fp32); wq_gu [E][2 m][d] int8 (the
    gate rows, then the up rows) with scales s_gu [E][2 m]; wq_down [E][d][m]
    int8 with scales s_down [E][d]; bias [E] fp32 or None; factor [E] fp32 or None
    (the ACE table of the skip rule); router_bias [E] fp32 or None, part of the logits
    (bias takes part in the choice alone).  d is a multiple of 64, m of 16, neither above
    16384; E <= 512, k <= 16.  Contiguous tensors on one device, gamma and the weights
    from 16-byte boundaries.  gate: the remaining arguments of ``ace.ace_gate_topk``
    (score, n_groups, topk_groups, group_score, renorm, scale)."""

    def __init__(self, gamma, w_router, wq_gu, s_gu, wq_down, s_down, k, max_tokens, bias=None,
                 factor=None, eps=1e-6, gate=None, router_bias=None):
        E, m2, d = wq_gu.shape
        m = m2 // 2
        if m2 % 2 or tuple(wq_down.shape) != (E, d, m) or tuple(w_router.shape) != (E, d):
            raise ValueError("wq_gu [E][2 m][d], wq_down [E][d][m] and w_router [E][d] do not match")
        if d % 64 or m % 16:
            raise ValueError("d must be a multiple of 64 and m of 16, are %d and %d" % (d, m))
        if max_tokens < 1 or not 1 <= k <= E:
            raise ValueError("max_tokens must be positive and 1 <= k <= E")
        if k > 16 or E > 512 or max(d, m) > 16384 or max_tokens * k > ace.MAX_COUNT:
            raise ValueError("k <= 16, E <= 512, d and m <= 16384 and max_tokens * k <= %d are served" % ace.MAX_COUNT)
        if not eps >= 0:
            raise ValueError("eps must not be negative")
        dev = w_router.get_device()
        for t, name, dtype, shape in ((wq_gu, "wq_gu", torch.int8, (E, m2, d)), (s_gu, "s_gu", torch.float32, (E, m2)),
                                      (wq_down, "wq_down", torch.int8, (E, d, m)),
                                      (s_down, "s_down", torch.float32, (E, d)),
                                      (bias, "bias", torch.float32, (E,)), (factor, "factor", torch.float32, (E,)),
                                      (router_bias, "router_bias", torch.float32, (E,))):
            if t is None and name[0] == "s":
                raise TypeError("%s is missing" % name)
            ace.check_arg(t, name, dev, dtype, shape)
        for t, name in ((gamma, "gamma"), (w_router, "w_router"), (wq_gu, "wq_gu"), (wq_down, "wq_down")):
            if t.data_ptr() % 16:
                raise ValueError("%s must start on a 16-byte boundary" % name)
        ace.check_gate(E, k, **(gate or {}))
        self.gamma, self.bias, self.factor, self.eps = gamma, bias, factor, float(eps)
        self.wq_gu, self.s_gu, self.wq_down, self.s_down = wq_gu, s_gu, wq_down, s_down
        self.w_router, self.router_bias, dtype = w_router, router_bias, w_router.dtype
        self.router = ace.make_router_layer(gamma, w_router, router_bias)
        if dev < 0:
            raise ValueError("LayerI8: tensors must be on a CUDA device")
        self.E, self.d, self.m, self.k, self.max_tokens, self.dtype = E, d, m, int(k), int(max_tokens), dtype
        self.gate, self.dev = dict(gate or {}), dev
        dev, T, S = gamma.device, int(max_tokens), int(max_tokens) * int(k)
        i32, f32, i8 = (dict(dtype=t, device=dev) for t in (torch.int32, torch.float32, torch.int8))
        self.xq, self.xs = torch.empty(T, d, **i8), torch.empty(T, **f32)
        self.sum, self.logits = torch.empty(T, d, dtype=dtype, device=dev), torch.empty(T, E, **f32)
        self.idx, self.weight = torch.empty(S, **i32), torch.empty(S, **f32)
        self.keep = torch.empty(S, dtype=torch.uint8, device=dev)
        self.offsets, self.slot_of = torch.empty(E + 1, **i32), torch.empty(S, **i32)
        self.slot_token, self.slot_gate = torch.empty(S, **i32), torch.empty(S, **f32)
        self.gu = torch.empty(S, 2 * m, dtype=dtype, device=dev)
        self.hq, self.hs = torch.empty(S, m, **i8), torch.empty(S, **f32)
        self.yslot = torch.empty(S, d, dtype=dtype, device=dev)
        # a workspace a call, so that each keeps its status word
        self.ws = [ace.alloc_workspace(ace.ace_logits_workspace_size(self.router, T), dev)] + \
            [ace.alloc_workspace(256, dev) for _ in range(3)]
        for w in self.ws:
            w.zero_()  # status() before the first call
        self.tokens, self.views = 0, None
        # the stream of the buffers' last use, and the end of that use
        self.lock, self.here, self.done = threading.Lock(), torch.cuda.current_stream(dev), torch.cuda.Event()
        self.done.record(self.here)

    def forward(self, u, y, residual=None, sum=None, tau=0.0, stream=None):
        """y [T][d] = the layer's output for u [T][d] (+ residual; sum, if given,
        receives u + residual, and may be either of them).  Slots but a token's
        largest are skipped where weight * factor < tau.  T <= max_tokens.  Rows of
        u and residual may lie apart and start anywhere; y and sum are contiguous,
        from 16-byte boundaries, and apart from each other; y may be u or residual."""
        T, tau = u.shape[0], float(tau)
        if u.dim() != 2 or T > self.max_tokens or u.shape[1] != self.d or u.dtype != self.dtype:
            raise ValueError("u must be [T <= %d][%d] %s" % (self.max_tokens, self.d, self.dtype))
        if u.get_device() != self.dev:
            raise ValueError("u must be on the layer's device")
        if y.shape != u.shape or y.dtype != u.dtype or y.get_device() != self.dev:
            raise ValueError("y must have u's shape, dtype and device")
        if not y.is_contiguous() or (sum is not None and not sum.is_contiguous()):
            raise ValueError("y and sum must be contiguous")
        if y.data_ptr() % 16 or (sum is not None and sum.data_ptr() % 16):
            raise ValueError("y and sum must start on 16-byte boundaries")
        if sum is not None and abs(sum.data_ptr() - y.data_ptr()) < y.numel() * y.element_size():
            raise ValueError("y and sum overlap")
        if stream is not None and stream.device.index != self.dev:
            raise ValueError("stream must be on the layer's device")
        if T == 0:
            return y
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.forward(u, y, residual, sum, tau)
        if self.dev != torch.cuda.current_device():
            with torch.cuda.device(u.device):
                return self.forward(u, y, residual, sum, tau)
        with self.lock:
            if torch.cuda.is_current_stream_capturing():
                self._enqueue(u, y, residual, sum, tau)
                return y
            if ace.current_raw_stream(self.dev) != self.here.cuda_stream:
                self.here = torch.cuda.current_stream()
                self.here.wait_event(self.done)
            try:
                self._enqueue(u, y, residual, sum, tau)
            finally:
                self.done.record(self.here)
        return y

    def _views(self, T):
        """The buffers' parts that T tokens use."""
        k, S = self.k, T * self.k
        idx, weight, keep, slot_of = (t[:S].view(T, k) for t in (self.idx, self.weight, self.keep, self.slot_of))
        return (self.xq[:T], self.xs[:T], self.logits[:T], self.sum[:T], idx, weight, keep, slot_of,
                self.slot_token[:S], self.slot_gate[:S], self.gu[:S], self.hq[:S], self.hs[:S], self.yslot[:S],
                self.offsets[self.E:])

    def _enqueue(self, u, y, residual, sum, tau):
        if u.shape[0] != self.tokens:  # as many as the call before: a decode loop
            self.tokens, self.views = u.shape[0], self._views(u.shape[0])
        xq, xs, logits, own_sum, idx, weight, keep, slot_of, slot_token, slot_gate, gu, hq, hs, yslot, n = self.views
        if sum is None and (residual is not None or not u.is_contiguous() or u.data_ptr() % 16):
            sum = own_sum  # the router reads whole rows in 16-byte vectors
        ace.ace_add_rmsnorm(u, self.gamma, residual=residual, sum=sum, q=xq, q_scale=xs, eps=self.eps)
        ace.ace_moe_logits(self.router, u if sum is None else sum, logits, self.ws[0], eps_rms=self.eps)
        ace.ace_gate_topk(logits, idx, weight, bias=self.bias, factor=self.factor, tau=tau, keep=keep,
                          **self.gate)
        ace.ace_moe_group(idx, self.E, self.offsets, slot_of, keep=keep, gate=weight, slot_token=slot_token,
                          slot_gate=slot_gate)
        ace.ace_matmul_i8(xq, xs, self.wq_gu, self.s_gu, gu, self.ws[1], offsets=self.offsets, row_of=slot_token)
        ace.ace_swiglu(gu, q=hq, q_scale=hs, n_valid=n)
        ace.ace_matmul_i8(hq, hs, self.wq_down, self.s_down, yslot, self.ws[2], offsets=self.offsets,
                          slot_scale=slot_gate)
        ace.ace_moe_combine(slot_of, yslot, y, self.ws[3])

    def status(self, stream=None):
        """(code, flags) of the last call, the first of its steps that is not
        ACE_OK (synchronises; of a replay on another stream, name it)."""
        with torch.cuda.device(self.ws[0].device):
            self.done.synchronize()
            codes = [ace.ace_read_status(w, stream) for w in self.ws]
        return next((c for c in codes if c[0] != ace.ACE_OK), codes[-1])
