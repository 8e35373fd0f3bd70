"""One MoE layer's expert computation in training, driven through the C ABI.

``MoeLayerBuffers`` owns every device buffer of the path (torch allocations,
sized once from the host capacities) and ``forward`` / ``backward`` enqueue the
library calls in order on one stream -- (router logits,) route, dispatch,
grouped SwiGLU forward, combine; then optionally compaction, backward dx (+ dg),
dW and the router's backward.  No step here computes anything itself: every
value comes from libmoe's kernels.  ``MoeBlockBuffers`` puts the layer into its
block the same way: layer norm, router with scored routing, routed experts, and
a gated shared expert whose last product adds the routed sum.  ``MoeHeadBuffers``
(the vocabulary loss) and ``AdamWBuffers`` (the optimizer's states) make a training
step of it: block forward, head forward and backward, block backward, AdamW.
"""
from __future__ import annotations

import dataclasses

import torch

from . import moe


@dataclasses.dataclass(frozen=True)
class ScoredRouting:
    """How moe_route_scored chooses and weighs (its arguments of these names)."""
    score: int = moe.MOE_SCORE_SIGMOID
    n_groups: int = 1
    top_groups: int = 1
    group_top: int = 1
    renormalize: bool = True
    scale: float = 1.0


@dataclasses.dataclass(frozen=True)
class BalanceLoss:
    """A balance loss of weight alpha over n_seq sequences of the batch (moe_balance_loss_fwd)."""
    alpha: float
    n_seq: int = 1


class MoeLayerBuffers:
    def __init__(self, T, H, F, E, k, dtype=torch.bfloat16, device="cuda", rho=None, dw=True, dg=True,
                 router=False, keep_graph=True, quota_cap=None, gather_rows=None, overlap_dw=False, routing=None,
                 balance=None):
        """rho: quota ratio of the compacted backward (None: no compaction);
        quota_cap: the per-expert quota directly (e.g. from
        moe.moe_quota_cap_for_budget), instead of rho.  keep_graph=False: the
        forward keeps no pre-activations [hg|hu]; the backward recomputes them
        from the token rows (the recompute path that pull request #44 keeps
        behind keep_graph=False).  gather_rows: every GEMM reads the token
        rows x and the saved activations through the pair / row indices
        (perm, kept_perm, kept_src), so neither x_sorted nor the compacted
        copies are materialized; False materializes them (moe_dispatch's row
        copy, moe_compact_pairs' row gathers).  Results are the same bit for
        bit.  None picks gathering unless dW runs over all pairs: there the
        weight-gradient GEMM streams each expert's x rows many times, and
        contiguous rows serve it better than one copy costs.  overlap_dw: the
        weight gradients run on a second stream (default priority) alongside
        the dX GEMM and the dx sum, from the point where the dx call signals dO
        and dh complete (moe_signal_dh_ready); the caller's stream then waits
        for them.  Results are the same bit for bit.  routing: a ScoredRouting;
        tokens are then routed by scores (moe_route_scored) instead of by the
        softmax over the selected logits.  balance: a BalanceLoss (of a layer with
        its router): the forward leaves balance_loss [1] with balance_counts and
        balance_mean [n_seq, E], the backward adds its gradient to the logits'."""
        self.routing, self.balance = routing, balance
        self.T, self.H, self.F, self.E, self.k = T, H, F, E, k
        self.keep_graph = keep_graph
        self.N = N = T * k
        self.dtype, self.rho, self.dw, self.want_dg = dtype, rho, dw, dg
        dev = torch.device(device)
        self.device = dev
        self.overlap_dw = bool(overlap_dw) and dw
        if self.overlap_dw:
            self._dw_stream = torch.cuda.Stream(device=dev)  # default priority
            self._dh_ready = torch.cuda.Event()
            self._dh_ready.record(torch.cuda.current_stream(dev))  # creates the underlying hipEvent
        i32, f32 = torch.int32, torch.float32
        em = lambda *s, dt=dtype: torch.empty(*s, dtype=dt, device=dev)  # noqa: E731
        self.topk_idx = em(T, k, dt=i32)
        self.topk_w = em(T, k, dt=f32)
        self.counts = em(E, dt=i32)
        self.offsets = em(E + 1, dt=i32)
        self.perm = em(N, dt=i32)
        self.inv_perm = em(N, dt=i32)
        ws = moe.moe_dispatch_workspace_bytes(T, E, k)
        self.ws = em(max(ws, 16), dt=torch.uint8)
        compacted = rho is not None or quota_cap is not None
        self.gather_rows = (compacted or not dw) if gather_rows is None else bool(gather_rows)
        self.x_sorted = None if self.gather_rows else em(N, H)
        self.h_save = em(N, 2 * F)
        self.a_save = em(N, F)
        self.o_sorted = em(N, H)
        self.y = em(T, H)
        self.quota_cap = quota_cap
        self.compacted = rho is not None or quota_cap is not None
        if self.compacted:
            cap = moe.moe_quota_cap(T, E, k, rho) if quota_cap is None else quota_cap
            self.R = min(N, E * cap)
            self.kept_counts = em(E, dt=i32)
            self.kept_offsets = em(E + 1, dt=i32)
            self.kept_perm = em(self.R, dt=i32)
            self.kept_src = em(self.R, dt=i32)
            self.kept_inv = em(N, dt=i32)
            g = self.gather_rows
            self.x_kept = None if g else em(self.R, H)
            self.a_kept = None if g or not dw else em(self.R, F)
            # pre-activations of the kept rows: recomputed into it, or (materialized) gathered
            self.h_kept = em(self.R, 2 * F) if (not keep_graph or not g) else None
            self.score = em(N, dt=f32)
        else:
            self.R = N
        R = self.R
        self.dO = em(R, H)
        self.dh = em(R, 2 * F)
        self.dX = em(R, H)
        self.dx = em(T, H)
        self.dg = em(T, k, dt=f32) if dg else None
        if dw:
            self.dw_gate = em(E, H, F)
            self.dw_up = em(E, H, F)
            self.dw_down = em(E, F, H)
        self.router = router
        if router:  # logits = x W_r in front of routing; its backward needs dg
            assert dg, "the router backward needs dg"
            self.logits = em(T, E, dt=f32)
            self.dlogits = em(T, E, dt=f32)
            self.dw_r = em(H, E)
            self.router_ws = em(max(moe.moe_router_workspace_bytes(T, H, E), 16), dt=torch.uint8)
        if balance is not None:
            assert router, "the balance loss needs the router"
            S = balance.n_seq
            self.balance_counts = em(S, E, dt=i32)
            self.balance_mean, self.balance_loss = em(S, E, dt=f32), em(1, dt=f32)
            self.balance_ws = em(max(moe.moe_balance_loss_workspace_bytes(T, E, S), 16), dt=torch.uint8)

    # ------------------------------------------------------------------ forward
    def _balance_args(self, stream):
        score = self.routing.score if self.routing is not None else moe.MOE_SCORE_SOFTMAX
        return dict(score=score, alpha=self.balance.alpha, seq_offsets=self._seq_offsets, stream=stream)

    def forward(self, logits, x, w_gate, w_up, w_down, stream=None, w_r=None, wq=None, wt=None, route_bias=None,
                seq_offsets=None):
        """With w_r (a layer built with router=True) the logits are x W_r and
        the `logits` argument is ignored.  With wq (moe.Fp8Weights of the same
        frozen weights) the expert GEMMs read the fp8 copy.  With wt
        (moe.Fp8KMajorWeights) both expert GEMMs run on the fp8 matrix cores:
        the token rows are quantized per row, then gathered on load.
        route_bias: the selection bias [E] of a layer with `routing`.
        seq_offsets: where the balance loss' sequences lie, [n_seq + 1]."""
        assert self.balance is None or w_r is not None, "the balance loss needs the router's logits"
        assert self.balance is not None or seq_offsets is None, "sequences are the balance loss'"
        self._x = x  # the backward reads token rows through the pair ids
        self._seq_offsets = seq_offsets
        if w_r is not None:
            moe.moe_router_fwd(x, w_r, self.logits, self.router_ws, stream)
            logits = self.logits
        if self.routing is not None:
            moe.moe_route_scored(logits, route_bias, self.topk_idx, self.topk_w, self.k,
                                 **dataclasses.asdict(self.routing), stream=stream)
        else:
            assert route_bias is None, "a selection bias needs a layer with scored routing"
            moe.moe_route_topk(logits, self.topk_idx, self.topk_w, self.k, stream)
        if self.balance is not None:
            moe.moe_balance_loss_fwd(logits, self.topk_idx, self.balance_counts, self.balance_mean, self.balance_loss,
                                     self.balance_ws, **self._balance_args(stream))
        g = self.gather_rows or wt is not None  # index-only dispatch: the forward gathers x rows itself
        moe.moe_dispatch(self.topk_idx, None if g else x, self.counts, self.offsets, self.perm, self.inv_perm,
                         None if g else self.x_sorted, self.ws, self.E, stream)
        if wt is not None:
            if not hasattr(self, "xq"):
                dev, u8, f32 = self.device, torch.uint8, torch.float32
                self.xq = torch.empty(self.T, self.H, dtype=u8, device=dev)
                self.x_scale = torch.empty(self.T, dtype=f32, device=dev)
                self.aq = torch.empty(self.N, self.F, dtype=u8, device=dev)
                self.a_scale = torch.empty(self.N, dtype=f32, device=dev)
            moe.moe_quantize_rows_fp8(x, self.xq, self.x_scale, stream)
            moe.moe_grouped_swiglu_fwd_fp8(self.offsets, self.xq, self.x_scale, wt,
                                           self.h_save if self.keep_graph else None, self.a_save, self.aq,
                                           self.a_scale, self.o_sorted, self.N, perm=self.perm, k=self.k,
                                           stream=stream)
        elif wq is not None:
            assert self.keep_graph, "the fp8 path keeps the pre-activations"
            moe.moe_grouped_swiglu_fwd_fp8w(self.offsets, x if g else self.x_sorted, wq, self.h_save, self.a_save,
                                            self.o_sorted, self.N, perm=self.perm if g else None, k=self.k,
                                            stream=stream)
        elif self.gather_rows:
            moe.moe_grouped_swiglu_fwd_gather(self.offsets, x, self.perm, w_gate, w_up, w_down,
                                              self.h_save if self.keep_graph else None, self.a_save, self.o_sorted,
                                              self.k, self.N, max_expert_rows=self.T, stream=stream)
        else:
            moe.moe_grouped_swiglu_fwd(self.offsets, self.x_sorted, w_gate, w_up, w_down,
                                       self.h_save if self.keep_graph else None, self.a_save, self.o_sorted, self.N,
                                       max_expert_rows=self.T, stream=stream)
        moe.moe_combine(self.o_sorted, self.inv_perm, self.topk_w, self.y, self.k, stream)
        return self.y

    # ----------------------------------------------------------------- backward
    def compact(self, score, stream=None):
        """Selection within the quotas; index-only when rows are gathered on load."""
        kg, g = self.keep_graph, self.gather_rows
        moe.moe_compact_pairs(self.counts, self.offsets, self.perm, score, self.rho or 1.0, self.kept_counts,
                              self.kept_offsets, self.kept_perm, self.kept_src, self.kept_inv, self.T, self.k,
                              None if g else self.x_sorted, None if g or not self.dw else self.a_save,
                              None if g or not kg else self.h_save, None if g else self.x_kept,
                              None if g or not self.dw else self.a_kept, None if g or not kg else self.h_kept, stream,
                              cap=self.quota_cap)

    def backward(self, dy, w_gate, w_up, w_down, score=None, stream=None, w_r=None, wq=None, dbalance=None):
        """dx (+ dg) and, for full fine-tuning, dW.  With a quota the backward
        runs on the compacted retained pairs; score: a pair-indexed fp32 tensor,
        None (the routing weights) or "metric" (moe_pair_scores: the norm of
        each pair's rank-one dW_down term).  With w_r, the router's backward
        follows: dlogits, dw_r, and its share added to dx.  dbalance [1] fp32: the
        gradient that reaches the balance loss (None: 1), whose own joins the
        logits' there; a layer with a balance loss needs w_r."""
        assert dbalance is None or self.balance is not None, "no balance loss in this backward"
        assert self.balance is None or w_r is not None, "the balance loss' gradient needs the router's backward"
        g, k = self.gather_rows, self.k
        if self.compacted:
            if isinstance(score, str):
                assert score == "metric", score
                moe.moe_pair_scores(self.inv_perm, self.topk_w, self.a_save, dy, self.score, stream)
                score = self.score
            self.compact(self.topk_w.view(-1) if score is None else score, stream)
            offsets, inv, pairs, src = self.kept_offsets, self.kept_inv, self.kept_perm, self.kept_src
        else:
            offsets, inv, pairs, src = self.offsets, self.inv_perm, self.perm, None
        # rows of the backward: x, a and the pre-activations h, each either a
        # contiguous buffer or a source buffer read through a row map
        if g:
            x_rows, x_src, a_rows, a_src = self._x, pairs, self.a_save, src
        else:
            x_rows, x_src = (self.x_kept if self.compacted else self.x_sorted), None
            a_rows, a_src = (self.a_kept if self.compacted else self.a_save), None
        if not self.keep_graph:  # recompute [hg | hu] of the backward's rows
            h_rows, h_src = (self.h_kept if self.compacted else self.h_save), None
            moe.moe_grouped_swiglu_recompute(offsets, x_rows, w_gate, w_up, h_rows, None, self.R,
                                             max_expert_rows=self.T, stream=stream, x_src=x_src, x_div=k)
        elif self.compacted and not g:
            h_rows, h_src = self.h_kept, None
        else:
            h_rows, h_src = self.h_save, src
        extra = dict(inv_all=self.inv_perm if self.want_dg else None, o_sorted=self.o_sorted if self.want_dg else None,
                     dg=self.dg, stream=stream, h_src=h_src)
        if self.dw and self.overlap_dw:
            moe.moe_signal_dh_ready(self._dh_ready)
        if wq is not None:  # frozen fp8 weights: no weight gradient
            assert not self.dw, "fp8 weights are frozen: no dW"
            moe.moe_grouped_bwd_dx_fp8w(offsets, inv, dy, self.topk_w, h_rows, wq, self.dO, self.dh, self.dX,
                                        self.dx, self.R, **extra)
        else:
            moe.moe_grouped_bwd_dx(offsets, inv, dy, self.topk_w, h_rows, w_gate, w_up, w_down, self.dO, self.dh,
                                   self.dX, self.dx, self.R, **extra)
        if self.dw:
            # dW reads dO and dh only: on the side stream it runs alongside dX
            # and the dx sum, from the moment the dx call signals them complete
            s_main = stream if stream is not None else torch.cuda.current_stream(self.device)
            s_dw = self._dw_stream if self.overlap_dw else s_main
            if self.overlap_dw:
                s_dw.wait_event(self._dh_ready)
            moe.moe_grouped_bwd_dw(offsets, x_rows, a_rows, self.dO, self.dh, self.dw_gate, self.dw_up,
                                   self.dw_down, self.R, s_dw, x_src=x_src, x_div=k, a_src=a_src)
            if self.overlap_dw:
                s_main.wait_stream(s_dw)
        if w_r is not None and (self.routing is not None or self.balance is not None):
            # without scored routing: the softmax over the selected logits is the renormalised softmax over all
            r = self.routing or ScoredRouting(moe.MOE_SCORE_SOFTMAX)
            moe.moe_route_scored_bwd(self.logits, self.topk_idx, self.dg, self.dlogits, r.score, r.renormalize, r.scale,
                                     stream)
            if self.balance is not None:
                moe.moe_balance_loss_bwd(self.logits, self.balance_counts, self.dlogits, k, dloss=dbalance,
                                         dl_add=self.dlogits, **self._balance_args(stream))
            moe.moe_router_bwd_dlogits(self._x, w_r, self.dlogits, self.dw_r, self.dx, True, self.router_ws, stream)
        elif w_r is not None:
            moe.moe_router_bwd(self._x, w_r, self.topk_idx, self.topk_w, self.dg, self.dlogits, self.dw_r, self.dx,
                               True, self.router_ws, stream)
        return self.dx


class MoeBlockBuffers:
    """A MoE block over T tokens of width H, without its skip connection:

        xn = layernorm(x),  y = experts(route(xn W_r), xn) + (silu(xn S_gate) * (xn S_up)) S_down

    E routed experts of width F (top k, chosen by `routing`) and a shared gated
    expert of width S.  forward / backward take the parameters as a dict:
    gamma, beta (or None), w_r, w_gate, w_up, w_down, s_gate [H, S], s_up [H, S],
    s_down [S, H], and route_bias [E] (optional); backward leaves the gradients
    in `grads` under the same names (the selection bias has none)."""

    def __init__(self, T, H, F, E, k, S, routing=ScoredRouting(), dtype=torch.bfloat16, device="cuda", eps=1e-5,
                 balance=None):
        self.layer = L = MoeLayerBuffers(T, H, F, E, k, dtype, device, router=True, routing=routing, balance=balance)
        self.eps = eps
        em = lambda *s, dt=dtype: torch.empty(*s, dtype=dt, device=L.device)  # noqa: E731
        self.xn, self.y, self.dx = em(T, H), em(T, H), em(T, H)
        self.mean, self.rstd = em(T, dt=torch.float32), em(T, dt=torch.float32)
        self.up, self.z_gate, self.hidden = em(T, S), em(T, S), em(T, S)
        self.d_hidden, self.d_up, self.dz = em(T, S), em(T, S), em(T, S)
        need = max(moe.moe_layernorm_workspace_bytes(T, H), moe.moe_linear_workspace_bytes(T, H, S, dtype),
                   moe.moe_linear_workspace_bytes(T, S, H, dtype), 16)
        self.ws = em(need, dt=torch.uint8)  # of one call at a time: they follow each other on one stream
        self.grads = dict(gamma=em(H), beta=em(H), w_r=L.dw_r, w_gate=L.dw_gate, w_up=L.dw_up, w_down=L.dw_down,
                          s_gate=em(H, S), s_up=em(H, S), s_down=em(S, H))

    def forward(self, x, p, stream=None, seq_offsets=None):
        self._x = x
        moe.moe_layernorm_fwd(x, p["gamma"], p.get("beta"), self.xn, self.mean, self.rstd, self.eps, stream)
        routed = self.layer.forward(None, self.xn, p["w_gate"], p["w_up"], p["w_down"], stream, w_r=p["w_r"],
                                    route_bias=p.get("route_bias"), seq_offsets=seq_offsets)
        moe.moe_linear_fwd(self.xn, p["s_up"], None, self.up, workspace=self.ws, stream=stream)
        moe.moe_linear_fwd(self.xn, p["s_gate"], None, self.hidden, act=moe.MOE_ACT_SILU, mul=self.up,
                           z_save=self.z_gate, workspace=self.ws, stream=stream)
        moe.moe_linear_fwd(self.hidden, p["s_down"], None, self.y, residual=routed, workspace=self.ws, stream=stream)
        return self.y

    def backward(self, dy, p, dx_add=None, stream=None, dbalance=None):
        """dx (+ dx_add, the gradient that reaches x past the block) and `grads`;
        dbalance: as for MoeLayerBuffers.backward."""
        g, ws, s = self.grads, self.ws, stream
        dxn = self.layer.backward(dy, p["w_gate"], p["w_up"], p["w_down"], stream=stream, w_r=p["w_r"],
                                  dbalance=dbalance)
        moe.moe_linear_bwd(self.hidden, p["s_down"], dy, None, self.d_hidden, g["s_down"], workspace=ws, stream=s)
        moe.moe_linear_bwd(self.xn, p["s_gate"], self.d_hidden, self.dz, dxn, g["s_gate"], act=moe.MOE_ACT_SILU,
                           z=self.z_gate, mul=self.up, dmul=self.d_up, dx_add=dxn, workspace=ws, stream=s)
        moe.moe_linear_bwd(self.xn, p["s_up"], self.d_up, None, dxn, g["s_up"], dx_add=dxn, workspace=ws, stream=s)
        moe.moe_layernorm_bwd(self._x, p["gamma"], self.mean, self.rstd, dxn, self.dx, g["gamma"],
                              g["beta"] if p.get("beta") is not None else None, ws, dx_add, s)
        return self.dx


class MoeHeadBuffers:
    """The vocabulary loss over T tokens of width H: the head's weights [H, V], of
    whose columns the first `vocab` (None: all) are classes.  forward leaves loss and
    lse [T] and mean = {mean loss, 1 / counted tokens}; backward dx and, with dw, the
    weights' gradient."""

    def __init__(self, T, H, V, vocab=None, dtype=torch.bfloat16, device="cuda", dw=True):
        dev = torch.device(device)
        em = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device=dev)  # noqa: E731
        self.vocab = vocab
        self.loss, self.lse, self.mean = em(T), em(T), em(2)
        self.dx = em(T, H, dt=dtype)
        self.dw = em(H, V, dt=dtype) if dw else None
        self.ws = em(max(moe.moe_vocab_loss_workspace_bytes(T, H, V, dtype), 16), dt=torch.uint8)

    def forward(self, x, w, target, stream=None):
        moe.moe_vocab_loss_fwd(x, w, target, self.loss, self.lse, self.mean, self.ws, self.vocab, stream)
        return self.mean

    def backward(self, x, w, target, dloss=None, scale=1.0, stream=None):
        """Of scale times the mean loss, or with dloss [T] of scale times sum dloss loss."""
        moe.moe_vocab_loss_bwd(x, w, target, self.loss, self.lse, self.mean, self.dx, self.dw, self.ws, dloss, scale,
                               self.vocab, stream)
        return self.dx


class AdamWBuffers:
    """AdamW over named parameters and their gradients (of one dtype, which stay where
    they are): moments of `bits` 32 or 8 and, with `master`, fp32 copies of bf16
    parameters.  weight_decay: of all, or a dict by name (0 for those that are not in
    it).  lr [1] and counter live on the device, so a captured step takes each replay's
    rate and counts on.  The plan is made once, of the gradients' addresses: gradients
    that moved would need a new one (moe.AdamWPlan, 0.16 ms of the host's time for 64
    tensors and 0.8 for 400, beside a step of 8 us over 64 small ones)."""

    def __init__(self, params, grads, lr, weight_decay=0.0, betas=(0.9, 0.999), eps=1e-8, bits=32, master=False, seed=0):
        assert bits in (32, 8), f"moments of {bits} bits"
        self.betas, self.eps, self.seed = betas, eps, seed
        self.state, tensors = {}, []
        for name, p in params.items():
            dev, n = p.device, p.numel()
            decay = weight_decay.get(name, 0.0) if isinstance(weight_decay, dict) else weight_decay
            if bits == 8:
                z = lambda dt, n=n: torch.zeros(n, dtype=dt, device=dev)  # noqa: E731
                s = dict(m=z(torch.uint8), v=z(torch.uint8), m_scale=z(torch.float32, -(-n // 256)),
                         v_scale=z(torch.float32, -(-n // 256)))
            else:
                s = dict(m=torch.zeros_like(p, dtype=torch.float32), v=torch.zeros_like(p, dtype=torch.float32))
            if master:
                s["master"] = p.detach().to(torch.float32, copy=True)
            self.state[name] = s
            tensors.append(moe.AdamWTensor(p, grads[name], weight_decay=decay, **s))
        self.plan = moe.AdamWPlan(tensors)
        self.counter = torch.zeros(2, dtype=torch.int32, device=dev)
        self.lr = torch.full((1,), lr, dtype=torch.float32, device=dev)

    def step(self, grad_scale=None, stream=None):
        moe.moe_adamw_step(self.plan, self.counter, self.lr, *self.betas, self.eps, grad_scale, self.seed, stream)
