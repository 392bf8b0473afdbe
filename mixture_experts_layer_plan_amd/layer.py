"""Device buffers for one layer shape and the call sequence of one training step.

``LayerBuffers`` allocates (through torch, on the current device) every output,
the plan, the saved activations and the workspaces that the C-ABI asks for.
``run_layer`` enqueues [norm ->] [router projection ->] route [-> balance loss] -> plan ->
[MX weight quantisation ->] forward [-> adapters] [-> backward -> adapters' backward -> router
backward -> norm's backward -> AdamW step]
on the current stream.  Both only move pointers; the arithmetic is in libmoe.so.

Options of ``LayerBuffers`` beside the layer's shape:
  scoring      a ``binding.scoring``: route by moe_route_scored instead of moe_route, with
               the selection bias ``router_bias`` fp32 [E] of the inputs, if they hold one
  router_proj  the inputs hold ``w_router`` bf16 [E, H] instead of logits; its gradient is
               ``dw_router``, and dx includes the router's term (bf16 and MXFP8; the fp32
               layer has router_gemm)
  adapters     (n, rank): low-rank adapters of many requests beside the whole layer (bf16 and
               MXFP8), y = layer(x) + scale_a (x A_a^T) B_a^T.  The inputs hold ``lora_a`` bf16
               [n, rank, H], ``lora_b`` bf16 [n, H, rank], ``lora_scale`` fp32 [n] and
               ``adapter_idx`` int32 [T] (-1: no adapter); the gradients are ``d_lora_a`` and
               ``d_lora_b``.  y and dx are rounded to bf16 before the adapters' terms join
               them, and again after; dx a third time when the router's term joins it.
  norm         (kind, eps): the layer's input is the norm of ``x``, joined with ``residual``
               [T, H] if the inputs hold one, with the weight ``norm_w`` [H] and the bias
               ``norm_b`` [H] if they hold them.  The layer then reads ``xn``; ``h`` is the joined
               row (written only with a residual).  dx is the gradient of x and of residual alike
               and includes ``dh`` [T, H], what reaches h on the residual stream, if the inputs
               hold it (rounded to the element type before, as dx of the layer, and after);
               ``d_norm_w``, ``d_norm_b``
  balance      a ``binding.balance``: ``loss`` [1] and ``counts`` int32 [n_seq, E] of the routing,
               by sequences ``seq_start`` int32 [n_seq + 1] if the inputs hold them, and its
               gradient, times ``d_loss`` fp32 [1] if they hold one, in d_logits

``AdamW`` keeps the states of the weights that a set of inputs holds and updates them in
place from the gradients of the buffers; ``run_layer(..., adamw=a, hyper=h)`` ends with a step.
"""
from __future__ import annotations

import torch

from . import binding as B


class LayerBuffers:
    def __init__(self, T, H, I, E, k, I_shared=0, dtype="bf16", backward=True,
                 router_gemm=False, device="cuda", T_minibatch=0, replay=False,
                 fused_forward=False, scoring=None, router_proj=False, adapters=None,
                 norm=None, balance=None):
        if dtype not in ("bf16", "f32", "mxfp8"):
            raise ValueError(f"unsupported dtype {dtype}")
        if router_gemm and dtype != "f32":
            # the router GEMM calls take fp32 x and accumulate into an fp32 dx
            raise ValueError("router_gemm needs dtype 'f32'")
        if dtype == "f32" and (router_proj or adapters):
            raise ValueError("router_proj and adapters need dtype 'bf16' or 'mxfp8'")
        self.dtype = dtype
        self.dt = B.DTYPES[dtype]
        flags = (B.MOE_REPLAY if replay else 0) | (B.MOE_FUSED_FORWARD if fused_forward else 0)
        self.s = B.shape(T, H, I, E, k, I_shared, T_minibatch, flags)
        tdt = torch.float32 if dtype == "f32" else torch.bfloat16
        dev = torch.device(device)
        u8 = dict(dtype=torch.uint8, device=dev)
        self.tdt = tdt
        self.topk_idx = torch.empty((T, k), dtype=torch.int32, device=dev)
        self.topk_w = torch.empty((T, k), dtype=torch.float32, device=dev)
        self.plan = torch.empty(B.moe_plan_bytes(self.s), **u8)
        self.saved = torch.empty(B.moe_saved_bytes(self.s, self.dt), **u8)
        self.ws_fwd = torch.empty(B.moe_workspace_bytes(self.s, self.dt, False), **u8)
        self.wq = torch.empty(B.moe_mx_weights_bytes(self.s), **u8) if dtype == "mxfp8" else None
        self.wq_stale = False   # whether a step has changed the weights since wq was made
        self.y = torch.empty((T, H), dtype=tdt, device=dev)
        self.scoring = scoring
        self.router_proj = router_proj
        self.logits = (torch.empty((T, E), dtype=torch.float32, device=dev)
                       if router_gemm or router_proj else None)
        if router_proj:
            self.ws_router = torch.empty(max(B.moe_router_workspace_bytes(self.s, bw)
                                             for bw in (False, backward)), **u8)
        self.lora = None
        if adapters:
            n, r = adapters
            self.lora = B.lora_shape(T, H, H, n, r)
            self.lora_plan = torch.empty(B.moe_lora_plan_bytes(self.lora), **u8)
            self.lora_saved = (torch.empty(B.moe_lora_saved_bytes(self.lora), **u8)
                               if backward else None)
            self.ws_lora = torch.empty(max(B.moe_lora_workspace_bytes(self.lora, bw)
                                           for bw in (False, backward)), **u8)
            if backward:
                self.d_lora_a = torch.empty((n, r, H), dtype=tdt, device=dev)
                self.d_lora_b = torch.empty((n, H, r), dtype=tdt, device=dev)
        self.norm = None
        if norm:
            kind, eps = norm
            self.norm = B.norm_shape(T, H, kind, eps)
            self.xn = torch.empty((T, H), dtype=tdt, device=dev)
            self.h = torch.empty((T, H), dtype=tdt, device=dev)
            self.norm_stats = torch.empty((T, 2), dtype=torch.float32, device=dev)
            if backward:
                self.d_norm_w = torch.empty((H,), dtype=tdt, device=dev)
                self.d_norm_b = torch.empty((H,), dtype=tdt, device=dev)
                self.ws_norm = torch.empty(B.moe_norm_workspace_bytes(self.norm), **u8)
        self.balance = balance
        if balance is not None:
            n = balance.n_seq
            self.loss = torch.empty((1,), dtype=torch.float32, device=dev)
            self.counts = torch.empty((n, E), dtype=torch.int32, device=dev)
            self.balance_scales = torch.empty((n,), dtype=torch.float32, device=dev)
            self.ws_balance = torch.empty(B.moe_balance_workspace_bytes(self.s, balance), **u8)
        self.backward = backward
        if backward:
            self.ws_bwd = torch.empty(B.moe_workspace_bytes(self.s, self.dt, True), **u8)
            self.dx = torch.empty((T, H), dtype=tdt, device=dev)
            self.dw_gate = torch.empty((E, I, H), dtype=tdt, device=dev)
            self.dw_up = torch.empty((E, I, H), dtype=tdt, device=dev)
            self.dw_down = torch.empty((E, H, I), dtype=tdt, device=dev)
            if I_shared:
                self.ds_gate = torch.empty((I_shared, H), dtype=tdt, device=dev)
                self.ds_up = torch.empty((I_shared, H), dtype=tdt, device=dev)
                self.ds_down = torch.empty((H, I_shared), dtype=tdt, device=dev)
            else:
                self.ds_gate = self.ds_up = self.ds_down = None
            self.d_topk_w = torch.empty((T, k), dtype=torch.float32, device=dev)
            self.d_logits = torch.empty((T, E), dtype=torch.float32, device=dev)
            self.dw_router = (torch.empty((E, H), dtype=tdt, device=dev)
                              if router_gemm or router_proj else None)

    def plan_views(self) -> dict:
        return B.plan_views(self.s, self.plan)


def quantize_weights(b: LayerBuffers, inp: dict, stream=None):
    """MXFP8 weights in the six orientations the MX GEMMs read (once per weight update)."""
    B.moe_quantize_weights_mxfp8(b.s, inp["w_gate"], inp["w_up"], inp["w_down"], b.wq, stream)
    b.wq_stale = False


def run_forward(b: LayerBuffers, inp: dict, stream=None, quantize=True):
    """route -> plan -> forward; for MXFP8 also the weight quantisation unless
    ``quantize`` is False (weights already quantised into ``b.wq``) and no step of an
    ``AdamW`` over these buffers has changed them since."""
    s = b.s
    logits = _logits(b, inp)
    if b.norm is not None:
        res = inp.get("residual")
        fn = B.moe_norm_f32 if b.dtype == "f32" else B.moe_norm_bf16
        fn(b.norm, inp["x"], res, inp.get("norm_w"), inp.get("norm_b"), None if res is None else b.h,
           b.xn, b.norm_stats, stream)
    x = _x(b, inp)
    if "w_router" in inp:
        if b.logits is None:
            raise ValueError("inputs carry w_router but the buffers have no router GEMM")
        if b.router_proj:
            B.moe_router_logits_bf16(s, x, inp["w_router"], b.logits, b.ws_router, stream)
        else:
            B.moe_router_logits_f32(s, x, inp["w_router"], b.logits, stream)
    if b.scoring is not None:
        B.moe_route_scored(s, b.scoring, logits, inp.get("router_bias"), b.topk_idx, b.topk_w,
                           stream)
    else:
        B.moe_route(s, logits, b.topk_idx, b.topk_w, stream)
    if b.balance is not None:
        B.moe_balance_loss(s, b.balance, logits, b.topk_idx, inp.get("seq_start"), b.loss, b.counts,
                           b.balance_scales, b.ws_balance, stream)
    B.moe_plan(s, b.topk_idx, b.plan, stream)
    _run_experts(b, inp, stream, quantize)
    if b.lora is not None:
        B.moe_lora_plan(b.lora, inp["adapter_idx"], b.lora_plan, stream)
        B.moe_lora_bf16(b.lora, b.lora_plan, x, inp["lora_a"], inp["lora_b"],
                        inp["lora_scale"], b.y, b.y, b.lora_saved, b.ws_lora, stream)


def _logits(b: LayerBuffers, inp: dict):
    return b.logits if "w_router" in inp else inp["logits"]


def _x(b: LayerBuffers, inp: dict):
    return inp["x"] if b.norm is None else b.xn


def _run_experts(b: LayerBuffers, inp: dict, stream, quantize):
    s, x = b.s, _x(b, inp)
    if b.dtype == "mxfp8":
        if quantize or b.wq_stale:
            quantize_weights(b, inp, stream)
        B.moe_forward_mxfp8(s, b.plan, x, b.topk_w, b.wq, inp.get("s_gate"),
                            inp.get("s_up"), inp.get("s_down"), b.y, b.saved, b.ws_fwd, stream)
        return
    fwd = B.moe_forward_bf16 if b.dtype == "bf16" else B.moe_forward_f32
    fwd(s, b.plan, x, b.topk_w, inp["w_gate"], inp["w_up"], inp["w_down"],
        inp.get("s_gate"), inp.get("s_up"), inp.get("s_down"), b.y, b.saved, b.ws_fwd, stream)


def run_backward(b: LayerBuffers, inp: dict, stream=None):
    s, x = b.s, _x(b, inp)
    if b.dtype == "mxfp8":
        B.moe_backward_mxfp8(s, b.plan, x, b.topk_w, b.wq, inp.get("s_gate"),
                             inp.get("s_up"), inp.get("s_down"), b.saved, inp["dy"], b.dx,
                             b.dw_gate, b.dw_up, b.dw_down, b.ds_gate, b.ds_up, b.ds_down,
                             b.d_topk_w, b.ws_bwd, stream)
    else:
        bwd = B.moe_backward_bf16 if b.dtype == "bf16" else B.moe_backward_f32
        bwd(s, b.plan, x, b.topk_w, inp["w_gate"], inp["w_up"], inp["w_down"],
            inp.get("s_gate"), inp.get("s_up"), inp.get("s_down"), b.saved, inp["dy"], b.dx,
            b.dw_gate, b.dw_up, b.dw_down, b.ds_gate, b.ds_up, b.ds_down, b.d_topk_w, b.ws_bwd,
            stream)
    if b.lora is not None:
        B.moe_lora_backward_bf16(b.lora, b.lora_plan, x, inp["lora_a"], inp["lora_b"],
                                 inp["lora_scale"], b.lora_saved, inp["dy"], b.dx, b.dx, b.d_lora_a,
                                 b.d_lora_b, b.ws_lora, stream)
    if b.scoring is not None:
        B.moe_route_scored_backward(s, b.scoring, _logits(b, inp), b.topk_idx, b.d_topk_w,
                                    b.d_logits, stream)
    else:
        B.moe_route_backward(s, b.topk_idx, b.topk_w, b.d_topk_w, b.d_logits, stream)
    if b.balance is not None:
        B.moe_balance_loss_backward(s, b.balance, _logits(b, inp), b.topk_idx, inp.get("seq_start"),
                                    b.counts, b.balance_scales, inp.get("d_loss"), b.d_logits,
                                    b.d_logits, stream)
    if "w_router" in inp and b.router_proj:
        B.moe_router_backward_bf16(s, x, inp["w_router"], b.d_logits, b.dx, b.dw_router, b.dx,
                                   b.ws_router, stream)
    elif "w_router" in inp:
        B.moe_router_backward_f32(s, x, inp["w_router"], b.d_logits, b.dw_router, b.dx,
                                  stream)
    if b.norm is not None:
        res = inp.get("residual")
        fn = B.moe_norm_backward_f32 if b.dtype == "f32" else B.moe_norm_backward_bf16
        fn(b.norm, inp["x"] if res is None else b.h, inp.get("norm_w"), b.norm_stats, b.dx,
           inp.get("dh"), b.dx, b.d_norm_w if "norm_w" in inp else None,
           b.d_norm_b if "norm_b" in inp else None, b.ws_norm, stream)


# weights of the inputs, their gradients in the buffers, and whether they decay (norms and
# biases do not)
_WEIGHTS = [("w_gate", "dw_gate", True), ("w_up", "dw_up", True), ("w_down", "dw_down", True),
            ("s_gate", "ds_gate", True), ("s_up", "ds_up", True), ("s_down", "ds_down", True),
            ("w_router", "dw_router", True), ("lora_a", "d_lora_a", True),
            ("lora_b", "d_lora_b", True), ("norm_w", "d_norm_w", False),
            ("norm_b", "d_norm_b", False)]


class AdamW:
    """The states of the weights in ``inp`` that ``b`` has gradients for, and the table of
    the step over them.  Weights and states are updated in place: both have to stay where
    they are.  ``state`` holds, by the weight's name, m and v (zeros; for state_bits = 8 codes,
    with m_scale and v_scale) and, if ``master``, the fp32 master (the weight's value).  They and
    the table are written on the current stream."""

    def __init__(self, b: LayerBuffers, inp: dict, state_bits=32, master=False, weight_decay=0.1):
        if master and b.dtype == "f32":
            raise ValueError("fp32 weights are their own masters")
        if not b.backward:
            raise ValueError("the buffers have no gradients")
        self.state, tensors = {}, []
        for name, grad, decays in _WEIGHTS:
            if name not in inp or getattr(b, grad, None) is None:
                continue
            w = inp[name]
            n, dev = w.numel(), w.device
            t = {"m": torch.zeros(n, dtype=torch.uint8 if state_bits == 8 else torch.float32, device=dev)}
            t["v"] = torch.zeros_like(t["m"])
            if state_bits == 8:
                t["m_scale"] = torch.zeros((n + 31) // 32, dtype=torch.uint8, device=dev)
                t["v_scale"] = torch.zeros_like(t["m_scale"])
            if master:
                t["master"] = w.to(torch.float32)
            self.state[name] = t
            tensors.append(dict(t, param=w, grad=getattr(b, grad),
                                weight_decay=weight_decay if decays else 0.0))
        if not tensors:
            raise ValueError("no weight of the inputs has a gradient in the buffers")
        typ = "f32" if b.dtype == "f32" else "bf16"
        self.shape = B.adamw_shape(sum(t["grad"].numel() for t in tensors), len(tensors), typ, typ,
                                   master, state_bits)
        self.table = torch.empty(B.moe_adamw_table_bytes(self.shape), dtype=torch.uint8,
                                 device=tensors[0]["grad"].device)
        self._tensors = tensors     # the table holds their addresses
        self._buffers = b
        B.moe_adamw_table(self.shape, tensors, self.table)

    def step(self, hyper, stream=None):
        """``hyper``: a ``binding.adamw_hyper`` of this step, or a device tensor of the bytes
        of one (which a captured step reads anew at every replay).  The next forward of MXFP8
        buffers quantises the new weights; for other buffers over the same weights, and behind
        the replay of a captured step alone, this is the caller's to do."""
        B.moe_adamw_step(self.shape, self.table, hyper, stream)
        self._mark(self._buffers)

    def _mark(self, b):
        if b.dtype == "mxfp8" and {"w_gate", "w_up", "w_down"} & self.state.keys():
            b.wq_stale = True

    def check(self, b: LayerBuffers, inp: dict):
        """ValueError unless the step reads the gradients of ``b`` and updates weights of
        ``inp`` (the table holds addresses; weights that it leaves out stay as they are)."""
        def ptr(t):
            return None if t is None else t.data_ptr()
        mine = {n: (ptr(t["param"]), ptr(t["grad"])) for n, t in zip(self.state, self._tensors)}
        its = {n: (ptr(inp[n]), ptr(getattr(b, g))) for n, g, _ in _WEIGHTS
               if n in inp and getattr(b, g, None) is not None}
        bad = sorted(n for n in mine if mine[n] != its.get(n))
        if bad:
            raise ValueError(f"the step is over other weights or gradients than this call's: {bad}")


def run_layer(b: LayerBuffers, inp: dict, backward: bool = True, stream=None, quantize=True,
              adamw: AdamW | None = None, hyper=None):
    """``adamw`` is over weights of ``inp`` and their gradients in ``b`` (ValueError otherwise).
    ``quantize=False``: ``b.wq`` holds the MXFP8 weights as they are before the call and,
    with a step, as they are after it."""
    if (adamw is None) != (hyper is None):
        raise ValueError("a step takes adamw and hyper")
    if adamw is not None and not backward:
        raise ValueError("a step takes the gradients of the backward")
    if adamw is not None:
        adamw.check(b, inp)
    run_forward(b, inp, stream, quantize)
    if backward:
        run_backward(b, inp, stream)
    if adamw is not None:
        adamw.step(hyper, stream)
        adamw._mark(b)
        if b.wq_stale and not quantize:     # here, so that replays of a captured call do it too
            quantize_weights(b, inp, stream)
