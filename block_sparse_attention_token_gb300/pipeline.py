"""The whole hot path as one object with preallocated device buffers.

forward(): (optional) token norm and three-axis rotary positions of Q and K -> reorder
Q, K, V into tiles (the rotation happens in that pass) -> block scores -> Top-p/Top-k selection
-> (optional) head balancing over P virtual ranks and slack-aware augmentation
of the CSR -> (optional) dependency-aware placement of blocks on the P
partitions -> KV demand of P partitions (+ gather) -> block-sparse attention
-> O in raster order (written there by attention itself where the tcgen05
kernel runs, else by an inverse reorder). backward(): dO into tiles ->
attention backward -> dQ, dK, dV in raster order (likewise) -> (optional) inverse
rotation and norm backward, with the gradients of the norm's weights. With a token
mask, block pairs that see nothing of each other are masked before the selection and
leave its lists after it (balancing, augmentation, placement and the KV demand count the
others), and attention runs over the tokens that the mask lets through; a score cap
applies in attention alone. Every step is one
or more libsparsp kernels on the current stream, except that by default the
KV demand gather runs on a side
stream beside attention (the caller's stream waits for both); nothing here
allocates after construction. capture() records forward() (and, with a
backward, forward() + backward()) as one CUDA graph, for shapes where the
host's launches, not the kernels, set the pace.
"""
from __future__ import annotations

import dataclasses

import torch

from . import (EST_LOWRANK, EST_MEAN, PROF_SLOTS, Shape, attn_bwd, attn_fwd, attn_launches, attn_workspace_size, augment,
               augment_workspace_size, balance_heads, Balance, predictor_fit,
               attn_masked_bwd, attn_masked_compacts, attn_masked_fwd, attn_masked_workspace_size, LISTS_SEEN, MaskPlan,
               mask_csr, mask_scores, norm_bwd, norm_fwd, norm_rope_bwd, norm_rope_fwd, norm_rope_workspace_size,
               norm_workspace_size, rope as rope_turn, RopeTable,
               block_scores, block_scores_pooled, block_scores_workspace_size, kv_demand, kv_gather, lib, placement,
               placement_workspace_size, reorder, reorder_pool, select, select_workspace_size, DemandOut,
               OUT_RASTER, IN_RASTER, pool_means, _whole)


@dataclasses.dataclass
class QKNorm:
    """Token norm of Q and of K in a Pipeline: layer norm, or RMS norm with rms, over
    the H*d values of a token, or over each head's d values with per_head. Weights
    and biases are float32 [H*d] or [d], or None; they are read at every forward(). one_pass
    (with per_head and a rotation): norm and rotation of Q and K in one kernel, rounded once
    and not between the two."""
    q_weight: torch.Tensor | None = None
    k_weight: torch.Tensor | None = None
    q_bias: torch.Tensor | None = None
    k_bias: torch.Tensor | None = None
    eps: float = 1e-6
    rms: bool = False
    per_head: bool = False
    one_pass: bool = False


class Pipeline:
    def _attn_flags(self) -> int:
        seen = self.mask is not None and (self._attn_on_seen or self.augment)
        return self.flags | (OUT_RASTER if self.raster_out else 0) | (LISTS_SEEN if seen else 0)

    def kernels_per_forward(self) -> int:
        """Kernels forward() launches: norm of Q and K (2, or 1 with the rotation in one pass) when there is one, reorder x3
        (the rotation is in that pass; with raster inputs a rotation or pooling pass over Q and K
        each), pool + product, masked scores (1) and lists (3) under a mask, select x3 (count,
        scan, fill), predictor fitting x7 when enabled, balancing (1) and augmentation x14 (keys, slack, four
        histogram + digit passes, row counts, ties, scan, fill) when enabled, placement x2 (affinity, greedy) when
        enabled, demand x5 (counter reset, bitmap, scan, list, gather), attention with the order of its
        work (attn_launches), inverse reorder (none when attention writes raster O)."""
        gather = 1 if self.demand.kg is not None else 0
        scores = (2 if self.est == EST_LOWRANK else 1) if self.fused else 2
        place = 2 if self.owner is not None else 0
        bal = (1 if self.migrations is not None else 0) + (14 if self.augment else 0)
        # projection, two score products, gradient products, loss (partials, sum), weight gradients
        pred = 7 if self.predictor_lr is not None else 0
        tiles = (2 if self.norm is not None else 0) + (2 if self.raster_in else 3)
        if self.one_pass:
            tiles = 1 + (0 if self.raster_in else 1)
        masked = 4 if self.mask is not None else 0
        attn = attn_launches(self.shape, False, self.mask is not None, self.cap, self._attn_flags())
        return tiles + scores + masked + pred + 3 + bal + place + 4 + gather + attn + (0 if self.raster_out else 1)

    def kernels_per_backward(self) -> int:
        """Reorder of dO, attention (attn_launches), an inverse rotation or reorder of dQ and dK
        each (no reorder when the backward writes raster gradients) and an inverse reorder of dV
        (likewise), norm backward (gradient, weights' sums) of Q and K."""
        attn = attn_launches(self.shape, True, self.mask is not None, self.cap, self._attn_flags())
        if self.one_pass:   # gradient and weights' sums of Q and K, reorder of dV
            return 1 + attn + 2 + (0 if self.raster_out else 1)
        back = (2 if self.rope is not None or not self.raster_out else 0) + (0 if self.raster_out else 1)
        return 1 + attn + back + (4 if self.norm is not None else 0)

    def __init__(self, shape: Shape, estimator: str, top_p: float, k_floor: int, P: int, rank: int = 16,
                 gather: bool = True, flags: int = 0, backward: bool = False, device="cuda",
                 fused_estimation: bool = True, placement: bool = False, migrations: int | None = None,
                 augment: bool = False, predictor_lr: float | None = None, overlap_demand: bool = True,
                 raster_inputs: bool = False, norm: QKNorm | None = None, rope: RopeTable | None = None,
                 rope_pos: torch.Tensor | None = None, mask: MaskPlan | None = None, cap: float = 0.0):
        """overlap_demand: after the KV demand lists (bitmap, offsets, indices),
        run the demand gather on a low-priority side stream while attention runs
        on a high-priority one; the two only read the same K/V, and the
        gather's CTAs (no shared memory) fit beside the persistent attention
        CTAs. forward() returns after both on the caller's stream. migrations: balance
        heads over P virtual ranks with at most this many
        migrations (None: no balancing). augment: fill each rank's slack with
        extra blocks (on the balanced ranks, or the contiguous head split);
        attention then runs on the augmented CSR. predictor_lr: with the
        low-rank estimator, after the scores are taken, one fitting step of the
        predictor weights (updated in place) against the real block scores.
        raster_inputs (forward-only, tcgen05 shapes, fused estimation): no
        reorder pass; the tile means come from a pooling read of raster Q and
        K, and the demand gather and attention read the raster tensors
        themselves (each block one 5-D TMA box), so forward()'s inputs stay
        in use until attention and the gather have finished. norm: token norm of Q and
        K first; backward() then also reads forward()'s q and k, and leaves the
        weights' gradients in self.norm_grads. rope: three-axis rotary positions
        of Q and K (rope_pos: int32 [B, N, 3] table positions, default the grid). mask: a
        token mask; cap: a score cap; both need shapes of the tcgen05 kernels."""
        self.shape, self.top_p, self.k_floor, self.P, self.rank, self.flags = shape, top_p, k_floor, P, rank, flags
        self.est = EST_LOWRANK if estimator == "lowrank" else EST_MEAN
        self.fused = fused_estimation
        s = shape
        dt = s.torch_dtype
        dev = torch.device(device)
        blocked = (s.B, s.H, s.N, s.d)
        self.raster_in = raster_inputs
        self.norm, self.rope, self.rope_pos, self.mask, self.cap = norm, rope, rope_pos, mask, float(cap)
        raster = (s.B, s.N, s.H, s.d)
        self.one_pass = norm is not None and norm.one_pass
        if self.one_pass and (not norm.per_head or rope is None):
            raise ValueError("norm and rotation in one pass need a norm per head and a rotation")
        self.qn = self.kn = self.qr = self.kr = None       # normed, and normed and turned, raster Q and K
        if norm is not None and not self.one_pass:
            self.qn, self.kn = (torch.empty(raster, dtype=dt, device=dev) for _ in range(2))
            stat = raster[:3] if norm.per_head else raster[:2]
            self.norm_stats = [(None if norm.rms else torch.empty(stat, dtype=torch.float32, device=dev),
                                torch.empty(stat, dtype=torch.float32, device=dev)) for _ in range(2)]
        if rope is not None and raster_inputs:
            self.qr, self.kr = (torch.empty(raster, dtype=dt, device=dev) for _ in range(2))
        self.qb = self.kb = self.vb = None
        if not raster_inputs:
            self.qb, self.kb, self.vb = (torch.empty(blocked, dtype=dt, device=dev) for _ in range(3))
        self.o = torch.empty((s.B, s.N, s.H, s.d), dtype=dt, device=dev)
        self.lse = torch.empty((s.B, s.H, s.N), dtype=torch.float32, device=dev)
        self.scores = torch.empty((s.B, s.H, s.nb, s.nb), dtype=torch.float32, device=dev)
        self.ws_scores = torch.empty(max(block_scores_workspace_size(s, self.est, rank), 16), dtype=torch.uint8,
                                     device=dev)
        self.qmeans, self.kmeans = (torch.empty((s.B, s.H, s.nb, s.d), dtype=torch.float32, device=dev)
                                    for _ in range(2))
        import ctypes
        n = lib().sparsp_block_scores_pooled_workspace_size(ctypes.byref(s), self.est, rank)
        self.ws_pooled = torch.empty(max(n, 16), dtype=torch.uint8, device=dev)
        self.row_ptr = torch.empty(s.rows + 1, dtype=torch.int32, device=dev)
        self.col_idx = torch.empty(s.rows * s.nb, dtype=torch.int32, device=dev)
        self.ws_sel = torch.empty(max(select_workspace_size(s), 16), dtype=torch.uint8, device=dev)
        W = (s.nb + 31) // 32
        parts = s.B * s.H * P
        kg = vg = None
        if gather:
            kg = torch.empty((parts * s.nb, s.Bt, s.d), dtype=dt, device=dev)
            vg = torch.empty_like(kg)
        self.demand = DemandOut(torch.empty((s.B, s.H, P, W), dtype=torch.int32, device=dev),
                                torch.empty(parts + 1, dtype=torch.int32, device=dev),
                                torch.empty(parts * s.nb, dtype=torch.int32, device=dev), kg, vg,
                                torch.empty(4, dtype=torch.int64, device=dev))
        self.migrations, self.augment = migrations, augment
        self.predictor_lr = predictor_lr
        if predictor_lr is not None:
            if self.est != EST_LOWRANK or not fused_estimation:
                raise ValueError("predictor fitting needs the low-rank estimator with fused estimation")
            self.predictor_loss = torch.empty(s.H, dtype=torch.float32, device=dev)
            self.gwq, self.gwk = (torch.empty((s.H, s.d, rank), dtype=torch.float32, device=dev) for _ in range(2))
            self.ws_pred = torch.empty(max(lib().sparsp_predictor_workspace_size(ctypes.byref(s), rank), 16),
                                       dtype=torch.uint8, device=dev)
        # the tcgen05 forward takes O straight into raster order (64-token blocks with
        # d = 128 beyond 1,024 blocks run the portable kernel, which writes block
        # order only); the tcgen05 backward (the same shapes) also reads raster O
        # and writes raster dQ, dK, dV
        fwd_raster = (s.torch_dtype == torch.bfloat16 and not (flags & 2) and s.Bt in (64, 128)
                      and s.d in (64, 128) and not (s.Bt == 64 and s.d == 128 and s.nb > 1024))
        self.raster_out = fwd_raster
        if raster_inputs and (backward or not fwd_raster or not fused_estimation):
            raise ValueError("raster inputs need a forward-only step on the tcgen05 kernel with fused estimation")
        # the stage after which forward()'s raster inputs are no longer read
        self.inputs_read_mark = ("overlap" if overlap_demand and gather else "attn_fwd") if raster_inputs \
            else "reorder"
        masked = mask is not None or self.cap != 0.0
        if masked and not fwd_raster:
            raise ValueError("a token mask or a score cap needs a shape of the tcgen05 kernels")
        self._qk_in = None   # forward()'s q and k (read by the norm's backward)
        # the stage of backward() after which the step's raster inputs are no longer read
        self.grad_inputs_read_mark = "reorder_dout" if norm is None else "norm_bwd"
        self._o_fwd = None   # the buffer forward() last wrote O to (read by backward() when raster)
        # block-order O (and gradients) only where attention does not write raster rows
        self.ob = None if self.raster_out else torch.empty(blocked, dtype=dt, device=dev)
        self.overlap_demand = overlap_demand
        if overlap_demand:
            lo, hi = torch.cuda.Stream.priority_range()   # least, greatest
            self._attn_stream = torch.cuda.Stream(device=dev, priority=hi)
            self._demand_stream = torch.cuda.Stream(device=dev, priority=lo)
            self._selected = torch.cuda.Event()
        self.balance = None
        if migrations is not None or augment:
            if migrations is None:
                self.migrations = 0
            self.balance = Balance(
                torch.empty((s.B, s.H), dtype=torch.int32, device=dev),
                torch.empty((s.B, 2, P), dtype=torch.int64, device=dev),
                torch.empty(max(s.B, 4), dtype=torch.int32, device=dev))
        if augment:
            self.row_ptr_aug = torch.empty(s.rows + 1, dtype=torch.int32, device=dev)
            self.col_idx_aug = torch.empty(s.rows * s.nb, dtype=torch.int32, device=dev)
            self.added = torch.empty((s.B, P), dtype=torch.int64, device=dev)
            self.ws_aug = torch.empty(max(augment_workspace_size(s, P), 16), dtype=torch.uint8, device=dev)
        self.csr = (self.row_ptr, self.col_idx)   # the lists attention runs on
        self._lists_flag = 0
        if mask is not None:
            # the selected pairs that see something; attention runs on them where it would make
            # the same lists itself
            self.row_ptr_seen = torch.empty(s.rows + 1, dtype=torch.int32, device=dev)
            self.col_idx_seen = torch.empty(s.rows * s.nb, dtype=torch.int32, device=dev)
            self._attn_on_seen = attn_masked_compacts(s)
        self.owner = self.ws_place = None
        if placement:
            self.owner = torch.empty((s.B, s.nb), dtype=torch.int32, device=dev)
            self.ws_place = torch.empty(max(placement_workspace_size(s), 16), dtype=torch.uint8, device=dev)
        n_ws = attn_masked_workspace_size(s, backward) if masked else attn_workspace_size(s, backward)
        self.ws_attn = torch.empty(max(n_ws, 16), dtype=torch.uint8, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.prof = torch.zeros(PROF_SLOTS, dtype=torch.int64, device=dev)
        if backward:
            self.dob = torch.empty(blocked, dtype=dt, device=dev)
            self.dqb = self.dkb = self.dvb = None
            if not self.raster_out:
                self.dqb, self.dkb, self.dvb = (torch.empty(blocked, dtype=dt, device=dev) for _ in range(3))
            self.dq, self.dk, self.dv = (torch.empty((s.B, s.N, s.H, s.d), dtype=dt, device=dev)
                                         for _ in range(3))
            # gradients between attention and the inverse rotation, and between that and the norm
            self._g_attn = [torch.empty(raster, dtype=dt, device=dev) for _ in range(2)] \
                if self.raster_out and (norm is not None or rope is not None) else None
            self._g_rope = [torch.empty(raster, dtype=dt, device=dev) for _ in range(2)] \
                if norm is not None and not self.one_pass and (rope is not None or not self.raster_out) else None
            self.norm_grads = None
            if norm is not None:
                cols = s.d if norm.per_head else s.H * s.d
                mk = lambda: torch.empty(cols, dtype=torch.float32, device=dev)
                # {"q_weight", "k_weight"[, "q_bias", "k_bias"]}: written by every backward()
                self.norm_grads = {x: mk() for x in ("q_weight", "k_weight")}
                if not norm.rms or norm.q_bias is not None or norm.k_bias is not None:
                    self.norm_grads.update({x: mk() for x in ("q_bias", "k_bias")})
                n_ws = norm_rope_workspace_size(s, s.H) if self.one_pass else norm_workspace_size(s, norm.rms, norm.per_head)
                self.ws_norm = torch.empty(max(n_ws, 16), dtype=torch.uint8, device=dev)

    def forward(self, q, k, v, wq=None, wk=None, prof: bool = False, mark=None, out=None, before=None):
        """mark: optional callable(stage_name, stream=None) invoked after each
        stage is enqueued (used to record CUDA events; stream None is the
        current stream). With overlap_demand the overlapped stages are marked on
        their own streams, each preceded by a "<stage>:begin" mark, and the
        region they share by "overlap". out: optional raster output buffer
        (default: self.o). before: optional callable(name) invoked just before
        input "q", "k" or "v" is first read (e.g. to wait for its copy). All are
        contiguous raster tensors, but q and k that a norm or a rotation reads may be
        slices of a wider one (one stride between tokens); ValueError otherwise."""
        s = self.shape
        _whole(s, "v", v)
        _whole(s, "out", out, True)
        mark = mark or (lambda name, stream=None: None)
        before = before or (lambda name: None)
        def prepared(name, x, normed, stats, weight, bias, turned, blocked, means):
            """Norm, rotation and tile order of Q or K, as far as this pipeline does
            them; returns the tensor that attention reads."""
            before(name)
            if self.norm is not None:
                n = self.norm
                norm_fwd(s, x, weight, bias, n.eps, n.rms, n.per_head, out=normed, mean=stats[0], rstd=stats[1])
                x = normed
            means = means if self.fused else None
            if self.rope is not None:
                return rope_turn(s, self.rope, x, out=turned if self.raster_in else blocked,
                                 out_blocked=not self.raster_in, pos=self.rope_pos, means=means, status=self.status)
            if self.raster_in:   # the tile means alone: attention and the gather read the raster tensors
                pool_means(s, x, means)
                return x
            if self.fused:       # the tile means come out of the reorder pass itself
                reorder_pool(s, x, blocked, means)
            else:
                reorder(s, x, blocked)
            return blocked

        self._qk_in = (q, k) if self.norm is not None else None
        if self.one_pass:
            n, tiles = self.norm, not self.raster_in
            before("q")
            before("k")
            aq, ak = norm_rope_fwd(s, self.rope, q, k, n.q_weight, n.k_weight, n.q_bias, n.k_bias, n.eps, n.rms,
                                   self.rope_pos, self.qb if tiles else self.qr, self.kb if tiles else self.kr, tiles,
                                   self.qmeans if self.fused else None, self.kmeans if self.fused else None, self.status)
        else:
            n, st = self.norm or QKNorm(), self.norm_stats if self.norm is not None else (None, None)
            aq = prepared("q", q, self.qn, st[0], n.q_weight, n.q_bias, self.qr, self.qb, self.qmeans)
            ak = prepared("k", k, self.kn, st[1], n.k_weight, n.k_bias, self.kr, self.kb, self.kmeans)
        if not self.raster_in:
            before("v")
            reorder(s, v, self.vb)
        mark("reorder")
        if self.fused:
            block_scores_pooled(s, self.qmeans, self.kmeans, self.est, wq, wk, self.rank, out=self.scores,
                                ws=self.ws_pooled)
        else:
            block_scores(s, self.qb, self.kb, self.est, wq, wk, self.rank, out=self.scores, ws=self.ws_scores)
        if self.mask is not None:
            mask_scores(s, self.mask, self.scores)
        mark("scores")
        if self.predictor_lr is not None:
            predictor_fit(s, self.qmeans, self.kmeans, wq, wk, self.predictor_lr, self.rank, self.predictor_loss,
                          self.gwq, self.gwk, self.ws_pred)
            mark("predictor")
        select(s, self.scores, self.top_p, self.k_floor, self.row_ptr, self.col_idx, self.ws_sel, self.status)
        rp, ci = self.row_ptr, self.col_idx
        self.csr, self._lists_flag = (rp, ci), 0
        if self.mask is not None:
            rp, ci = mask_csr(s, self.mask, rp, ci, self.row_ptr_seen, self.col_idx_seen, self.status)
            if self._attn_on_seen or self.augment:
                self.csr, self._lists_flag = (rp, ci), LISTS_SEEN
        mark("select")
        if self.balance is not None:
            balance_heads(s, self.P, rp, self.migrations, out=self.balance)
            mark("balance")
        if self.augment:
            rp, ci, _ = augment(s, self.P, self.scores, rp, ci, self.balance.head_rank,
                                self.row_ptr_aug, self.col_idx_aug, self.added, self.ws_aug, self.status)
            self.csr = (rp, ci)
            mark("augment")
        if self.owner is not None:
            placement(s, self.P, rp, ci, self.owner, self.ws_place, self.status)
            mark("placement")
        o = self.o if out is None else out
        # attention output: raster O directly, or block order and an inverse reorder
        o_attn, aflags = (o, self.flags | OUT_RASTER) if self.raster_out else (self.ob, self.flags)
        av = self.vb
        if self.raster_in:
            before("v")
            av, aflags = v, aflags | IN_RASTER

        def attention(stream=None):
            p = self.prof if prof else None
            if self.mask is not None or self.cap:
                attn_masked_fwd(s, aq, ak, av, *self.csr, 0.0, self.cap, self.mask, o_attn, self.lse, self.ws_attn,
                                aflags | self._lists_flag, p, self.status, stream)
            else:
                attn_fwd(s, aq, ak, av, *self.csr, 0.0, o_attn, self.lse, self.ws_attn, aflags, p, self.status, stream)

        if self.overlap_demand and self.demand.kg is not None:
            # the lists (bitmap, offsets, indices) first, on this stream: they need a
            # little shared memory, which attention leaves none of; then the gather
            # (no shared memory) beside attention
            main = torch.cuda.current_stream()
            lists = dataclasses.replace(self.demand, kg=None, vg=None)
            kv_demand(s, self.P, rp, ci, out=lists, status=self.status, owner=self.owner)
            mark("kv_demand")
            hi, lo = self._attn_stream, self._demand_stream
            mark("overlap:begin")
            self._selected.record(main)
            hi.wait_event(self._selected)
            lo.wait_event(self._selected)
            with torch.cuda.stream(hi):   # enqueued first: the persistent CTAs take their SMs first
                mark("attn_fwd:begin", hi)
                attention(hi)
                mark("attn_fwd", hi)
            with torch.cuda.stream(lo):
                mark("kv_gather:begin", lo)
                kv_gather(s, self.P, self.demand, ak, av, status=self.status, stream=lo, raster=self.raster_in)
                mark("kv_gather", lo)
            main.wait_stream(hi)
            main.wait_stream(lo)
            mark("overlap")
        else:
            if self.raster_in and self.demand.kg is not None:
                lists = dataclasses.replace(self.demand, kg=None, vg=None)
                kv_demand(s, self.P, rp, ci, out=lists, status=self.status, owner=self.owner)
                kv_gather(s, self.P, self.demand, ak, av, status=self.status, raster=True)
            else:
                kv_demand(s, self.P, rp, ci, self.kb, self.vb, out=self.demand, status=self.status,
                          owner=self.owner)
            mark("kv_demand")
            attention()
            mark("attn_fwd")
        if not self.raster_out:
            reorder(s, self.ob, o, inverse=True)
            mark("reorder_out")
        self._o_fwd = o
        return o, self.lse

    def backward(self, dout, prof: bool = False, mark=None, outs=None, before=None):
        """outs: optional raster (dQ, dK, dV) output buffers (default: self.dq, self.dk, self.dv);
        before: optional callable("do") invoked just before dout is first read.
        With raster_out the backward reads O from the buffer the last forward()
        wrote it to, which must still hold it, and writes the gradients' raster
        rows itself. With a norm it reads forward()'s q and k, which must still hold
        their values, and writes the weights' gradients to self.norm_grads. dout and
        outs are contiguous, but dQ and dK that a rotation or a norm writes may be
        slices like forward()'s q and k."""
        s = self.shape
        _whole(s, "dout", dout)
        if outs is not None:
            for name, t in zip(("dq", "dk", "dv"), outs):
                if name == "dv" or self.rope is None and self.norm is None:
                    _whole(s, name, t)
        mark = mark or (lambda name: None)
        if before is not None:   # e.g. to wait for dout's copy
            before("do")
        reorder(s, dout, self.dob)
        mark("reorder_dout")
        rp, ci = self.csr
        dq, dk, dv = (self.dq, self.dk, self.dv) if outs is None else outs
        gq, gk = (dq, dk) if self.norm is None and self.rope is None else (self._g_attn or (None, None))
        p = self.prof if prof else None
        if self.raster_out:
            if self._o_fwd is None:
                raise RuntimeError("backward() needs a forward() first")
            args = (s, self.qb, self.kb, self.vb, self._o_fwd, self.lse, self.dob, rp, ci, 0.0)
            if self.mask is not None or self.cap:
                attn_masked_bwd(*args, self.cap, self.mask, gq, gk, dv, self.ws_attn,
                                self.flags | OUT_RASTER | self._lists_flag, p, self.status)
            else:
                attn_bwd(*args, gq, gk, dv, self.ws_attn, self.flags | OUT_RASTER, p, self.status)
            mark("attn_bwd")
        else:
            attn_bwd(s, self.qb, self.kb, self.vb, self.ob, self.lse, self.dob, rp, ci, 0.0,
                     self.dqb, self.dkb, self.dvb, self.ws_attn, self.flags, p, self.status)
            mark("attn_bwd")
            gq, gk = self.dqb, self.dkb
        # dQ and dK back through the rotation (and to raster order), then through the norm
        if self.one_pass:
            n, grads = self.norm, self.norm_grads
            names = ("q", "k")
            norm_rope_bwd(s, self.rope, gq, gk, *self._qk_in, n.q_weight, n.k_weight, n.eps, n.rms, self.rope_pos,
                          not self.raster_out, dq, dk, [grads[x + "_weight"] for x in names],
                          [grads.get(x + "_bias") for x in names], self.ws_norm, self.status)
            if not self.raster_out:
                reorder(s, self.dvb, dv, inverse=True)
                mark("reorder_grads")
            mark("norm_bwd")
            return dq, dk, dv
        g_in = (gq, gk)
        g_out = (dq, dk) if self.norm is None else (self._g_rope or g_in)
        for g, to in zip(g_in, g_out):
            if self.rope is not None:
                rope_turn(s, self.rope, g, out=to, inverse=True, in_blocked=not self.raster_out, out_blocked=False,
                          pos=self.rope_pos, status=self.status)
            elif not self.raster_out:
                reorder(s, g, to, inverse=True)
        if not self.raster_out:
            reorder(s, self.dvb, dv, inverse=True)
            mark("reorder_grads")
        if self.norm is not None:
            n, grads = self.norm, self.norm_grads
            for x, g, to, (mean, rstd), w, name in zip(self._qk_in, g_out, (dq, dk), self.norm_stats,
                                                       (n.q_weight, n.k_weight), ("q", "k")):
                norm_bwd(s, g, x, w, mean, rstd, n.rms, n.per_head, dx=to, dw=grads[name + "_weight"],
                         db=grads.get(name + "_bias"), ws=self.ws_norm)
            mark("norm_bwd")
        return dq, dk, dv

    def capture(self, q, k, v, wq=None, wk=None, dout=None) -> "GraphedStep":
        """A CUDA graph of one step on these device buffers: forward(q, k, v),
        and backward(dout) too when dout is given. replay() reruns the whole
        step with one launch on whatever the buffers hold at that moment (the
        caller refills them in place) and returns what the step returns. The
        step runs once eagerly on a side stream first, as graph capture wants;
        the buffers stay bound to the graph. The captured step runs the KV
        demand gather before attention on one stream: a graph does not keep the
        side streams' priorities, without which the gather beside attention
        takes the SMs attention needs."""
        def step():
            out = self.forward(q, k, v, wq=wq, wk=wk)
            return out if dout is None else out + self.backward(dout)
        overlap, self.overlap_demand = self.overlap_demand, False
        try:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step()
            torch.cuda.current_stream().wait_stream(side)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                outs = step()
        finally:
            self.overlap_demand = overlap
        return GraphedStep(graph, outs)


class GraphedStep:
    """A captured Pipeline step (Pipeline.capture)."""

    def __init__(self, graph, outs):
        self.graph = graph
        self.outs = outs

    def replay(self):
        """Runs the step on the current stream; returns the step's outputs
        (O, LSE[, dQ, dK, dV]) in the buffers the capture bound."""
        self.graph.replay()
        return self.outs

