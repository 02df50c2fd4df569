"""The residual block of a transformer around the BEAM-masked MoE layer, for
serving and for training, and the layer's experts in 4-bit floating point.

    n   = x r(x) w_in                                    block_enter
    y   = layer(n)                                       forward, or Mx4Experts
    out = a x + b s(gate_t) gate_c w_out y r(y)          block_exit
    n'  = out r(out) w_next                              ... in the same pass

The pages describe the layer alone and leave the residual and the balance loss
to its caller (a token whose candidates are all masked passes through the
residual; the news article on BEAM, §4, sums three training losses).  Every
step runs in the library's kernels (C ABI); this module only sequences the
calls on torch's current stream and owns the buffers between them.  Nothing
synchronises or allocates after construction, so a step can be captured into a
CUDA graph.
"""
from __future__ import annotations

import torch

from . import abi


def _empty(*shape, dtype=torch.float32, device=None):
    return torch.empty(shape, dtype=dtype, device=device)


def _same_device(what, first, *others):
    """The kernels take every buffer of a block to be on one device."""
    for t in others:
        if t is not None and t.device != first.device:
            raise abi.BeamError(1, f"{what}: tensors on {first.device} and {t.device}")


def _check_routers(what, W_gate, W_mask, E, d, t):
    abi._arg(what, "W_gate", W_gate, t, (E, d), None)
    abi._arg(what, "W_mask", W_mask, t, (E, d), None, True)


class Mx4Experts:
    """The layer's experts with weights and rows in MXFP4, for T tokens:
    routing and grouping as in the layer, the token rows and the SwiGLU
    activations quantised, both projections as grouped 4-bit products, the
    weighted combine in fp32.

    Wg, Wm (or None) [E, d] bf16; W1, W3 [E, I, d], W2 [E, d, I] (bf16 or f32)
    are quantised once; d and I are multiples of 128."""

    def __init__(self, T, d, E, I, K, renorm, Wg, Wm, W1, W3, W2, tau=0.5):
        _check_routers("Mx4Experts", Wg, Wm, E, d, torch.bfloat16)
        for name, W, shape in (("W1", W1, (E, I, d)), ("W3", W3, (E, I, d)), ("W2", W2, (E, d, I))):
            if W.shape != shape:
                raise abi.BeamError(1, f"Mx4Experts: {name} has to be of shape {shape}, got "
                                       f"{tuple(W.shape)}")
        _same_device("Mx4Experts", Wg, Wm, W1, W3, W2)
        self.T, self.d, self.E, self.I, self.K = T, d, E, I, K
        self.Wg, self.Wm = Wg, Wm
        dev = self.device = Wg.device
        self.dsc = abi.desc(T, d, E, I, K, "bf16", renorm, tau=tau)
        self.w1, self.w3 = (self._weights(W, E * I, d) for W in (W1, W3))
        self.w2 = self._weights(W2, E * d, I)
        N = self.rows = max(T * K, 1)
        u8, i32, bf16 = torch.uint8, torch.int32, torch.bfloat16
        self.up = abi.mx4_desc(N, E, I, d, swiglu=True, out="bf16")
        self.down = abi.mx4_desc(N, E, d, I, out="f32")
        # zeroed, as mx4's are: check() may come before a call has written its word
        self.ws = abi.alloc_workspace(self.dsc, dev).zero_()
        self.ws_up = abi.alloc_mx4_workspace(self.up, dev)
        self.ws_down = abi.alloc_mx4_workspace(self.down, dev)
        self.idx = _empty(T, K, dtype=i32, device=dev)
        self.w = _empty(T, K, device=dev)
        self.counts = _empty(E, dtype=i32, device=dev)
        self.pair = _empty(N, dtype=i32, device=dev)
        self.expert = _empty(N, dtype=i32, device=dev)
        self.kept = _empty(4, dtype=i32, device=dev)
        self.pair_pos = _empty(T, K, dtype=i32, device=dev)
        self.x_rows = _empty(N, d, dtype=bf16, device=dev)
        self.x4 = (_empty(N, d // 2, dtype=u8, device=dev), _empty(N, d // 32, dtype=u8, device=dev))
        self.h = _empty(N, I, dtype=bf16, device=dev)
        self.h4 = (_empty(N, I // 2, dtype=u8, device=dev), _empty(N, I // 32, dtype=u8, device=dev))
        self.y_rows = _empty(N, d, device=dev)

    def _weights(self, W, rows, cols):
        codes = _empty(rows, cols // 2, dtype=torch.uint8, device=self.device)
        scales = _empty(rows, cols // 32, dtype=torch.uint8, device=self.device)
        abi.mx4_quantize(W.reshape(rows, cols), codes, scales, tiled=True)
        return codes, scales

    def forward(self, x, out, logits=None):
        """out [T, d] (bf16) for x [T, d] (bf16); logits f32 [T, 2 E] or None,
        as abi.route's."""
        # the calls below take addresses: they see neither shapes nor devices
        dev, rows = abi._current_device(), (self.T, self.d)
        abi._arg("Mx4Experts", "x", x, torch.bfloat16, rows, dev)
        abi._arg("Mx4Experts", "out", out, torch.bfloat16, rows, dev)
        abi._arg("Mx4Experts", "logits", logits, torch.float32, (self.T, 2 * self.E), dev, True)
        _same_device("Mx4Experts", self.counts, x)
        if self.T == 0:
            return out
        abi.route(self.dsc, x, self.Wg, self.Wm, self.idx, self.w, self.counts, logits=logits,
                  workspace=self.ws)
        abi.ep_dispatch(self.dsc, 1, x, self.idx, self.counts, self.x_rows, self.pair, self.expert,
                        self.kept, self.pair_pos, self.ws)
        n = self.kept[:1]  # the kept rows: their number stays on the device
        abi.mx4_quantize(self.x_rows, *self.x4, n_rows=n)
        abi.mx4_expert_product(self.up, *self.x4, self.counts, *self.w1, self.h, self.ws_up,
                               w3_codes=self.w3[0], w3_scales=self.w3[1])
        abi.mx4_quantize(self.h, *self.h4, n_rows=n)
        abi.mx4_expert_product(self.down, *self.h4, self.counts, *self.w2, self.y_rows,
                               self.ws_down)
        abi.ep_combine(self.dsc, self.y_rows, self.idx, self.w, self.pair_pos, out)
        return out

    def check(self):
        """Device error words of the last forward (synchronises)."""
        if self.T > 0:
            abi.check(self.dsc, self.ws)
            abi.mx4_check(self.up, self.ws_up)
            abi.mx4_check(self.down, self.ws_down)


class MoeBlock:
    """One residual block over T tokens.

    W_gate, W_mask (or None) [E, d], W1, W3 [E, I, d], W2 [E, d, I]: the layer's;
    w_in [d]; w_out [d], gate_c [d] or None; all of `dtype`.  balance: the
    balance loss's coefficient (training; 0 leaves it out), over n_seq packed
    sequences; beta weighs the mask-score penalty.  experts: an Mx4Experts of
    the same T, d and E that takes the layer's place (serving, bf16).

    No shared experts: a block that has them calls abi.forward_shared between
    abi.block_enter and abi.block_exit itself, and gate_t gates all of y, not
    a shared branch alone."""

    def __init__(self, T, d, E, I, K, renorm, W_gate, W_mask, W1, W3, W2, w_in, w_out=None,
                 gate_c=None, dtype="bf16", tau=0.5, eps=1e-6, res_scale=1.0, branch_scale=1.0,
                 balance=0.0, n_seq=1, count_kept=False, beta=0.0, train=False, experts=None):
        if train and experts is not None:
            raise ValueError("4-bit experts have no gradients")
        dev, t = W_gate.device, torch.bfloat16 if dtype == "bf16" else torch.float32
        if experts is not None:
            if (experts.T, experts.d, experts.E) != (T, d, E) or t != torch.bfloat16:
                raise ValueError(f"bf16 experts of T, d, E = {experts.T}, {experts.d}, {experts.E} in a "
                                 f"{dtype} block of {T}, {d}, {E}")
            _same_device("MoeBlock", experts.counts, W_gate)
        else:  # the layer's calls take addresses: they see neither shapes nor devices
            _check_routers("MoeBlock", W_gate, W_mask, E, d, t)
            for name, W, shape in (("W1", W1, (E, I, d)), ("W3", W3, (E, I, d)),
                                   ("W2", W2, (E, d, I))):
                abi._arg("MoeBlock", name, W, t, shape, None)
            _same_device("MoeBlock", W_gate, W_mask, W1, W3, W2)
        self.T, self.d, self.E, self.dtype = T, d, E, dtype
        self.layer = (W_gate, W_mask, W1, W3, W2)
        self.w_in, self.w_out, self.gate_c = w_in, w_out, gate_c
        self.experts, self.beta, self.train = experts, beta, train
        self.dsc = abi.desc(T, d, E, I, K, dtype, renorm, tau=tau)
        self.block = abi.block_desc(T, d, dtype, eps=eps, res_scale=res_scale,
                                    branch_scale=branch_scale, accumulate=True)
        self.n = _empty(T, d, dtype=t, device=dev)
        self.y = _empty(T, d, dtype=t, device=dev)
        # zeroed: check() may come before a call has written its error word
        self.ws = abi.alloc_workspace(self.dsc, dev).zero_() if experts is None else None
        self.loss = torch.zeros(1, device=dev)
        self.bal = None
        if not train:
            return
        masked = W_mask is not None
        if balance:
            # logits as route writes them: 2 E wide, the mask's half with a mask
            self.bal = abi.balance_desc(T, E, K, n_seq=n_seq, logits_ld=2 * E, has_mask=masked,
                                        count_kept=count_kept, tau=tau, coef=balance)
            i32 = torch.int32
            self.bal_ws = abi.alloc_balance_workspace(self.bal, dev)
            self.route_ws = abi.alloc_workspace(self.dsc, dev).zero_()  # an error word of its own
            self.logits = _empty(T, 2 * E, device=dev)
            self.dlogits = _empty(T, E, device=dev)
            self.cand = _empty(n_seq, E, dtype=i32, device=dev)
            self.kept = _empty(n_seq, E, dtype=i32, device=dev) if masked else None
            self.prob = _empty(n_seq, E, device=dev)
            self.idx = _empty(T, K, dtype=i32, device=dev)
            self.w = _empty(T, K, device=dev)
            self.counts = _empty(E, dtype=i32, device=dev)
        self.bwd_ws = abi.alloc_backward_workspace(self.dsc, dev).zero_()
        self.block_ws = abi.alloc_block_workspace(self.block, dev)
        self.dres = _empty(T, d, dtype=t, device=dev)
        self.dy = _empty(T, d, dtype=t, device=dev)
        self.dn = _empty(T, d, device=dev)
        z = lambda w: None if w is None else torch.zeros(w.shape, device=dev)  # noqa: E731
        self.grads = dict(w_in=z(w_in), w_out=z(w_out), gate_c=z(gate_c), W_gate=z(W_gate),
                          W_mask=z(W_mask), W1=z(W1), W3=z(W3), W2=z(W2))

    def zero_grad(self):
        for g in self.grads.values():
            if g is not None:
                g.zero_()

    def forward(self, x, out, gate_t=None, w_next=None, n_next=None, seq_begin=None):
        """out [T, d], and with w_next n_next [T, d].  When training with a
        balance loss, self.loss and the counts are those of this batch
        (seq_begin: its sequences); x and out are read again by backward."""
        abi.block_enter(self.block, x, self.w_in, self.n)
        if self.experts is not None:
            self.experts.forward(self.n, self.y)
        elif self.T > 0:
            abi.forward(self.dsc, self.n, *self.layer, self.y, self.ws)
        if self.bal is not None:
            if self.T > 0:
                abi.route(self.dsc, self.n, self.layer[0], self.layer[1], self.idx, self.w,
                          self.counts, logits=self.logits, workspace=self.route_ws)
            abi.balance(self.bal, self.logits, self.loss, self.cand, self.bal_ws,
                        kept_counts=self.kept, mean_prob=self.prob, seq_begin=seq_begin)
        abi.block_exit(self.block, x, self.y, out, w_out=self.w_out, gate_c=self.gate_c,
                       gate_t=gate_t, w_next=w_next, n_next=n_next)
        return out

    def backward(self, x, out, dout, dx, gate_t=None, dgate_t=None, w_next=None, dn_next=None,
                 dw_next=None, seq_begin=None, dloss=None):
        """dx [T, d] for the upstream gradient dout [T, d] (and dn_next f32
        [T, d] of the next norm's rows) of the last forward; the weights'
        gradients are added to self.grads and dw_next (f32).  dloss f32 [1]:
        the gradient of self.loss (1 if left out)."""
        if not self.train:
            raise ValueError("the block was made for serving")
        g = self.grads
        abi.block_exit_backward(self.block, self.y, dout, self.dres, self.dy, self.block_ws,
                                out=out, dn_next=dn_next, w_out=self.w_out, gate_c=self.gate_c,
                                gate_t=gate_t, w_next=w_next, dw_out=g["w_out"],
                                dgate_c=g["gate_c"], dgate_t=dgate_t, dw_next=dw_next)
        dlogits = None
        if self.bal is not None:
            counts = self.kept if self.bal.count_kept else self.cand
            abi.balance_backward(self.bal, self.logits, counts, self.dlogits, seq_begin=seq_begin,
                                 dloss=dloss)
            dlogits = self.dlogits
        if self.T > 0:
            abi.backward(self.dsc, self.n, *self.layer, self.dy, self.beta, self.dn, g["W_gate"],
                         g["W_mask"], g["W1"], g["W3"], g["W2"], self.bwd_ws, dlogits=dlogits)
        abi.block_enter_backward(self.block, x, self.w_in, self.dn, dx, g["w_in"], self.block_ws,
                                 dskip=self.dres)
        return dx

    def check(self):
        """Device error words of the last calls (synchronises)."""
        if self.experts is not None:
            self.experts.check()
        elif self.T > 0:
            abi.check(self.dsc, self.ws)
        if self.train and self.T > 0:
            abi.check(self.dsc, self.bwd_ws)
            if self.bal is not None:
                abi.check(self.dsc, self.route_ws)
