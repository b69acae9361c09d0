"""One GPU's share of a sharded optimizer step, driven through the C ABI.

``ShardRun`` holds, in HBM, everything one rank needs for a step of its shard
(per FSDP unit when there are several): the N_d ranks' gradient slices of
every micro-batch (the other ranks are simulated as extra buffers on this
GPU), the fp32 master/m/v shard, the fp32 reduced gradient (clip path, or
the micro-batch accumulator), the bf16 all-gather buffer (or the rank's own
bf16 shard) and the fp64 squared norm.  Inputs come from the seeded
generator, written directly into device memory.  ``step()`` issues exactly
the library calls of one optimizer step on one stream:

* no clip:   zero_shard_step(grad_slices=...)                 per unit
* clip:      shard_grad_sqnorm(...)                 (one unit), or
             shard_grad_sqnorm_units(...)           (all FSDP units at once)
             (squared norms summed in unit order: the global norm of the
             FSDP model; the other ranks' shards enter as other_sqnorm),
             then zero_shard_step(mean_in=..., sqnorm=...)    per unit
* fp32 slices, token weights or several micro-batches:
             shard_grad_reduce(micro=j, ...) for j = 0..m-1   per unit
             (the norm on the last micro-batch only), then
             zero_shard_step(mean_in=..., sqnorm=...)         per unit

``TableRun`` is a training step of the tied vocabulary table as a unit of its
own, its gradients made by the library's table operators instead of the
generator: every simulated rank looks its tokens up, is held to a teacher's
top logits, and leaves the table's gradient; then every rank's shard is
reduced, weighted by the ranks' valid tokens, clipped and updated.  Parameters
of the model between that are too small to shard (``whole``) are kept on every
rank, tensor by tensor; their norm joins the shards'.

``RelposBias`` is the position-bias table's call in such a model, with its
gradient.
"""
from __future__ import annotations

import math
from dataclasses import dataclass

import torch

import zsgen
from zsgen.workloads import (STREAM_EXP_AVG, STREAM_EXP_AVG_SQ, STREAM_MASTER, Workload,
                             grad_key, grad_stream)

from . import (ZS_F32, ZS_GRAD_BF16, ZS_GRAD_F32, ZS_OUT_GATHER, ZS_OUT_SHARD, adamw,
               distill_loss_grad, embed_grad, embed_lookup, make_distill, make_embed, make_reduce,
               make_tensors, relpos_bias, relpos_bias_grad, shard_grad_reduce, shard_grad_sqnorm,
               shard_grad_sqnorm_units, shard_pack_gather, tensors_clip, tensors_sqnorm,
               zero_shard_step, zs_distill_workspace_bytes, zs_embed_workspace_bytes, zs_layout,
               zs_relpos_workspace_bytes, zs_workspace_bytes, zs_workspace_bytes_units)


def _empty(n, dtype, device):
    # never a zero-size allocation: keeps every pointer non-NULL and aligned
    return torch.empty(max(int(n), 8), dtype=dtype, device=device)


@dataclass
class Unit:
    slices: torch.Tensor       # [m, n_d, pitch] int16 (bf16) or float32: micro-batch
                               # j, row r = rank r's slice, V elements used
    w: torch.Tensor
    m: torch.Tensor
    v: torch.Tensor
    mean: torch.Tensor | None
    out: torch.Tensor          # int16 [n_d*S] (gather) or [S] (shard)


class ShardRun:
    def __init__(self, wl: Workload, rank: int | None = None, device: str = "cuda",
                 units: int | None = None, store_mean: bool | None = None):
        self.wl = wl
        self.rank = wl.rank if rank is None else rank
        self.units = wl.units if units is None else units
        self.device = device
        out_mode = ZS_OUT_GATHER if wl.out_mode == "gather" else ZS_OUT_SHARD
        self.shard = zs_layout(wl.psi, wl.n_d, self.rank, wl.align, wl.stage, out_mode)
        self.clip = wl.max_grad_norm > 0
        self.micro = wl.micro_batches
        # fp32 slices, token weights and micro-batches go through the general
        # reduction, which always stores the reduced (accumulated) gradient
        self.general = wl.grad_dtype != "bf16" or bool(wl.rank_tokens) or self.micro > 1
        # the clip needs the norm before any update: store the mean, read it back
        self.store_mean = (self.clip or self.general) if store_mean is None else store_mean
        if self.general and not self.store_mean:
            raise ValueError("the general reduction needs the stored-gradient schedule")
        self.f32_grads = wl.grad_dtype == "f32"
        self.gsize = 4 if self.f32_grads else 2
        S, V, nd = self.shard.shard_len, self.shard.valid_len, wl.n_d
        out_len = nd * S if out_mode == ZS_OUT_GATHER else S
        if wl.stage == 0 and out_mode == ZS_OUT_GATHER:
            out_len = S
        self.out_len = out_len
        # Rows of the simulated ranks' slices start on a 128-byte boundary
        # (256 for fp32), as separately allocated per-rank buffers would; the
        # shard length itself need not be a multiple of 64 (the 70B shard's
        # 1,093,750,000 is not), and rows S elements apart would then start
        # off a cache-line boundary.
        self.slice_pitch = -(-S // 64) * 64
        self.units_data = []
        for _ in range(self.units):
            self.units_data.append(Unit(
                slices=torch.empty((self.micro, nd, self.slice_pitch),
                                   dtype=torch.float32 if self.f32_grads else torch.int16,
                                   device=device),
                w=_empty(V, torch.float32, device), m=_empty(V, torch.float32, device),
                v=_empty(V, torch.float32, device),
                mean=_empty(V, torch.float32, device) if self.store_mean else None,
                out=torch.empty(out_len, dtype=torch.int16, device=device)))
        # FSDP units of one layout: one clip-pass call for all of them
        self.grouped_units = self.units > 1 and not self.general
        wsb = (zs_workspace_bytes_units(self.shard, self.units) if self.grouped_units
               else zs_workspace_bytes(self.shard))
        self.workspace = torch.empty(wsb // 8, dtype=torch.float64, device=device)
        self.sqnorm = torch.zeros(1, dtype=torch.float64, device=device)
        self.t = wl.t0
        self.reduce_specs = [make_reduce(ZS_GRAD_F32 if self.f32_grads else ZS_GRAD_BF16, j,
                                         self.micro, wl.rank_tokens or None)
                             for j in range(self.micro)]

    # ---- inputs ------------------------------------------------------------------

    @property
    def V(self):
        return self.shard.valid_len

    @property
    def has_reduce_pass(self):
        """A separate reduction pass runs before the update: for the clip (the
        norm must be known first) and whenever the reduced gradient is stored."""
        return self.clip or self.store_mean

    def fill_state(self, out_fill: int | None = None):
        wl, V, off = self.wl, self.V, self.shard.shard_offset
        for u, d in enumerate(self.units_data):
            if V > 0:
                zsgen.dev_f32(d.w[:V], wl.seed, STREAM_MASTER, u, 0, wl.master_sigma, off)
                if wl.m_sigma is None:
                    d.m.zero_()
                else:
                    zsgen.dev_f32(d.m[:V], wl.seed, STREAM_EXP_AVG, u, 0, wl.m_sigma, off)
                if wl.v_sigma is None:
                    d.v.zero_()
                else:
                    zsgen.dev_f32(d.v[:V], wl.seed, STREAM_EXP_AVG_SQ, u, 0, wl.v_sigma, off,
                                  absval=True)
            if out_fill is not None:
                d.out.fill_(out_fill)

    def fill_grads(self, t: int):
        """Draw every micro-batch's slices of optimizer step t."""
        wl, V, off = self.wl, self.V, self.shard.shard_offset
        if V == 0:
            return
        for u, d in enumerate(self.units_data):
            for j in range(self.micro):
                key = grad_key(t, j, self.micro)
                for r in range(wl.n_d):
                    if self.f32_grads:
                        zsgen.dev_f32(d.slices[j, r, :V], wl.seed, grad_stream(u), r, key,
                                      wl.grad_sigma, off)
                    else:
                        zsgen.dev_bf16(d.slices[j, r, :V], wl.seed, grad_stream(u), r, key,
                                       wl.grad_sigma, off, p_out=wl.outlier_p,
                                       sigma_out=wl.outlier_sigma)

    # ---- the step -------------------------------------------------------------------

    def hparams(self, t: int):
        wl = self.wl
        return adamw(lr=wl.lr, beta1=wl.beta1, beta2=wl.beta2, eps=wl.eps,
                     weight_decay=wl.weight_decay, step=t, max_grad_norm=wl.max_grad_norm)

    def slice_ptrs(self, d: Unit, j: int = 0):
        base = d.slices[j].data_ptr()
        return [base + self.gsize * self.slice_pitch * r for r in range(self.wl.n_d)]

    def reduce_pass(self, stream=None):
        if self.grouped_units:
            ptrs = [p for d in self.units_data for p in self.slice_ptrs(d)]
            means = [d.mean for d in self.units_data] if self.store_mean else None
            shard_grad_sqnorm_units(self.shard, ptrs, means, self.workspace, self.sqnorm,
                                    stream=stream)
            return
        for u, d in enumerate(self.units_data):
            if not self.general:
                shard_grad_sqnorm(self.shard, self.slice_ptrs(d), d.mean, self.workspace,
                                  self.sqnorm, accumulate=u > 0, stream=stream)
                continue
            for j in range(self.micro):
                norm = self.clip and j == self.micro - 1
                shard_grad_reduce(self.shard, self.reduce_specs[j], self.slice_ptrs(d, j),
                                  d.mean, self.workspace if norm else None,
                                  self.sqnorm if norm else None, accumulate=u > 0,
                                  stream=stream)

    def update_pass(self, t: int, other_sqnorm: float = 0.0, stream=None):
        h = self.hparams(t)
        for d in self.units_data:
            if self.store_mean:
                zero_shard_step(self.shard, h, mean_in=d.mean,
                                sqnorm=self.sqnorm if self.clip else None,
                                other_sqnorm=other_sqnorm, master=d.w, exp_avg=d.m,
                                exp_avg_sq=d.v, param_out=d.out, stream=stream)
            else:
                zero_shard_step(self.shard, h, grad_slices=self.slice_ptrs(d),
                                sqnorm=self.sqnorm if self.clip else None,
                                other_sqnorm=other_sqnorm, master=d.w, exp_avg=d.m,
                                exp_avg_sq=d.v, param_out=d.out, stream=stream)

    def step(self, t: int | None = None, other_sqnorm: float = 0.0, stream=None):
        """Enqueue one optimizer step of every unit at bias-correction step t."""
        t = self.t if t is None else t
        if self.has_reduce_pass:
            self.reduce_pass(stream)
        self.update_pass(t, other_sqnorm, stream)
        self.t = t + 1

    # ---- bytes the step must move (algorithmic, per step) -------------------------------

    def algorithmic_bytes(self):
        """(reduce-pass bytes, update-pass bytes) over all units.

        reduce pass: N_d bf16 reads + fp32 mean write = 2 N_d + 4 B/param
        (fp32 slices: 4 N_d; micro-batch j > 0 also reads the accumulator)
        update pass: mean read (or N_d bf16 reads) + 12 B state read + 12 B
        state write + 2 B bf16 write; pads are written too (2 B each)."""
        nd, V, S = self.wl.n_d, self.V, self.shard.shard_len
        pads = S - V
        if self.general:
            # micro-batch j reads its slices, reads the accumulator (j > 0)
            # and writes it
            red = sum((self.gsize * nd + (4 if j > 0 else 0) + 4) * V for j in range(self.micro))
            upd = (4 + 12 + 12 + 2) * V + 2 * pads
        elif self.clip and self.store_mean:
            red = (2 * nd + 4) * V
            upd = (4 + 12 + 12 + 2) * V + 2 * pads
        elif self.clip:
            red = 2 * nd * V
            upd = (2 * nd + 26) * V + 2 * pads
        else:
            red = 0
            upd = (2 * nd + 26) * V + 2 * pads
        return red * self.units, upd * self.units


def _room(shape, dtype, n, device):
    """Memory of a gradient of `shape` of which a call writes n elements; others (a
    table's unused rows, the end of a flat buffer) are 0."""
    make = torch.empty if math.prod(shape) == n else torch.zeros
    return make(shape, dtype=dtype, device=device)


class RelposBias(torch.autograd.Function):
    """RelposBias.apply(r, table, scores, key_lengths, query_starts): relpos_bias
    of make_relpos's r (pitches without gaps), differentiable in table and
    scores; scores None: the bias alone, [batch, heads, queries, keys].  Scores and
    table may be of any shape relpos_bias takes; gradients are of the same."""

    @staticmethod
    def forward(ctx, r, table, scores=None, key_lengths=None, query_starts=None):
        shape = (r.batch, r.heads, r.queries, r.keys)
        dtype = torch.float32 if r.dtype == ZS_F32 else torch.bfloat16
        out = torch.empty(shape, dtype=dtype, device=table.device)
        relpos_bias(r, table.contiguous(), out, None if scores is None else scores.contiguous(),
                    key_lengths, query_starts)
        # the caller may change r before the backward pass
        ctx.r = type(r).from_buffer_copy(r)
        ctx.scores = scores.shape if scores is not None and ctx.needs_input_grad[2] else None
        # of the table the gradient needs no value: it may be written between the passes
        ctx.table = table.shape, table.dtype
        ctx.save_for_backward(key_lengths, query_starts)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        key_lengths, query_starts = ctx.saved_tensors
        dtable = _room(*ctx.table, ctx.r.buckets * ctx.r.heads, grad.device)
        dscores = None
        if ctx.scores is not None:
            dscores = _room(ctx.scores, grad.dtype, grad.numel(), grad.device)
        workspace = torch.empty(zs_relpos_workspace_bytes(ctx.r), dtype=torch.uint8,
                                device=grad.device)
        relpos_bias_grad(ctx.r, grad.contiguous(), dtable, workspace, dscores, key_lengths,
                         query_starts)
        return None, dtable, dscores, None, None


@dataclass
class TableBatch:
    """One rank's micro-batch: T token ids, the teacher's entries and the
    labels of its T positions (int64 on the GPU; -100: not trained on), and
    how many labels count, which the program that made them knows: the rank's
    mean is over them, and they weigh the rank.  (The distillation counts its
    rows on the device; at alpha = 1 a labelled row without a teacher entry has
    loss 0 and is in `valid` but not in `counted`.)"""
    ids: torch.Tensor              # int64 [T]
    teacher_ids: torch.Tensor      # int64 [T, k]
    teacher_logits: torch.Tensor   # float32 [T, k]
    labels: torch.Tensor           # int64 [T]
    valid: int


class TableRun:
    """The tied vocabulary table [rows, dim] as a ZeRO/FSDP unit of n_d ranks,
    all of them simulated here: each holds its shard of the fp32 state, and
    its own full gradient of the unit, of which every shard takes a slice.

    step(): per rank   embed_lookup, body, logits = hidden table^T,
                       distill_loss_grad, the head's gradient (a matrix
                       product, set), body's gradient, embed_grad (added)
            per shard  shard_grad_reduce(rank_tokens=valid tokens), the
                       squared norms summed
            per shard  zero_shard_step into its slot of the gathered table,
                       from which the next step looks up.

    f32_grads: the type in which a rank's gradient of the table is held, added
    to and reduced.  The head's matrix product itself is one of bf16 operands
    and leaves its kernel rounded to bf16, as a mixed-precision program's
    products do; embed_grad adds to it in fp32.

    body: a differentiable function of the hidden states [T, dim] that stands
    for the model between the two uses of the table; None: the identity.

    whole: parameters of body (fp32 initial values; body is required then, and is
    called with their bf16 copies behind the hidden states) that every rank keeps
    whole.  Their gradients, tensor by tensor, are averaged over the ranks by valid
    tokens (the all-reduce's stand-in), their squared norm is added to the shards',
    and the same coefficient clips them into the flat fp32 gradient of their own
    step:
            tensors_sqnorm(accumulate), tensors_clip, zero_shard_step (stage 0)

    max_grad_norm: the global norm's limit; <= 0: no clip, of shards and whole
    parameters alike.
    """

    def __init__(self, rows: int, dim: int, n_d: int, tokens: int, k: int, scale: float = 1.0,
                 temperature: float = 1.0, alpha: float = 1.0, f32_grads: bool = True, body=None,
                 lr: float = 1e-3, weight_decay: float = 0.01, max_grad_norm: float = 1.0,
                 whole=(), device: str = "cuda"):
        whole = list(whole)
        if whole and body is None:
            raise ValueError("whole parameters are the body's: a body is required")
        self.rows, self.dim, self.n_d, self.tokens = rows, dim, n_d, tokens
        self.body, self.f32_grads = body, f32_grads
        self.lr, self.weight_decay, self.max_grad_norm = lr, weight_decay, max_grad_norm
        self.shards = [zs_layout(rows * dim, n_d, r, 8, 3) for r in range(n_d)]
        S = self.shards[0].shard_len
        self.gather = torch.zeros(n_d * S, dtype=torch.bfloat16, device=device)
        self.table = self.gather[:rows * dim].view(rows, dim)
        grad_dtype = torch.float32 if f32_grads else torch.bfloat16
        self.grads = torch.zeros((n_d, n_d * S), dtype=grad_dtype, device=device)
        self.state = [[torch.zeros(max(s.valid_len, 8), device=device) for _ in range(3)]
                      for s in self.shards]                    # master, exp_avg, exp_avg_sq
        self.mean = [torch.empty(max(s.valid_len, 8), device=device) for s in self.shards]
        self.sqnorm = torch.zeros(1, dtype=torch.float64, device=device)
        self.reduce_ws = torch.empty(zs_workspace_bytes(self.shards[0]), dtype=torch.uint8,
                                     device=device)
        self.hidden = torch.empty((tokens, dim), dtype=torch.bfloat16, device=device)
        self.logits = torch.empty((tokens, rows), dtype=torch.bfloat16, device=device)
        self.dlogits = torch.empty_like(self.logits)
        self.dhidden = torch.empty_like(self.hidden)
        self.loss = torch.empty((n_d, tokens), device=device)
        self.loss_sum = torch.zeros(1, device=device)
        self.counted = torch.zeros(1, dtype=torch.int64, device=device)
        self.look = make_embed(tokens, rows, dim, scale=scale)
        self.back = make_embed(tokens, rows, dim, scale=scale,
                               table_dtype=ZS_F32 if f32_grads else 0)
        self.embed_ws = torch.empty(max(zs_embed_workspace_bytes(self.back), 16),
                                    dtype=torch.uint8, device=device)
        self.targets = make_distill(tokens, rows, k, temperature=temperature, alpha=alpha)
        self.distill_ws = torch.empty(zs_distill_workspace_bytes(self.targets), dtype=torch.uint8,
                                      device=device)

        self.whole = []
        if whole:
            self._keep_whole(whole, device)

    def _keep_whole(self, values, device):
        numel = [v.numel() for v in values]
        self.whole_shard = s = zs_layout(sum(numel), 1, 0, 8, 0)     # stage 0: all of it
        self.whole_state = [torch.zeros(max(s.valid_len, 8), device=device) for _ in range(3)]
        self.whole_gather = torch.zeros(s.shard_len, dtype=torch.bfloat16, device=device)
        self.whole_mean = torch.empty(max(s.valid_len, 8), device=device)

        def views(flat):
            return [p.view(v.shape) for p, v in zip(flat[:sum(numel)].split(numel), values)]

        for w, v in zip(views(self.whole_state[0]), values):
            w.copy_(v)
        shard_pack_gather(s, self.whole_state[0], self.whole_gather)
        self.whole = views(self.whole_gather)                         # what body reads
        # each rank's gradients, and their mean as an all-reduce leaves it
        self.rank_grads = [[torch.zeros_like(w) for w in self.whole] for _ in range(self.n_d)]
        self.whole_grads = [torch.zeros(w.shape, device=device) for w in self.whole]
        self.whole_list = make_tensors(self.whole_grads, views(self.whole_mean))

    def load(self, table: torch.Tensor):
        """Set the fp32 master table [rows, dim] and publish its bf16 copy."""
        flat = table.reshape(-1)
        for s, (w, _, _) in zip(self.shards, self.state):
            w[:s.valid_len] = flat[s.shard_offset:s.shard_offset + s.valid_len]
            shard_pack_gather(s, w, self.gather)

    def grad_table(self, r: int) -> torch.Tensor:
        return self.grads[r, :self.rows * self.dim].view(self.rows, self.dim)

    def rank_pass(self, r: int, b: TableBatch):
        """Rank r's forward and backward pass: its gradient and row losses."""
        embed_lookup(self.look, b.ids, self.table, self.hidden)
        if self.body is None:
            out = self.hidden
        else:
            leaf = self.hidden.detach().requires_grad_()
            kept = [w.detach().requires_grad_() for w in self.whole]
            out = self.body(leaf, *kept)
        h = out.detach()
        torch.mm(h, self.table.t(), out=self.logits)
        # the gradient of the rank's mean loss over its valid tokens
        self.targets.scale = 1.0 / max(b.valid, 1)
        distill_loss_grad(self.targets, self.logits, b.teacher_ids, b.teacher_logits,
                          self.loss[r], self.dlogits, labels=b.labels, loss_sum=self.loss_sum,
                          counted=self.counted, accumulate=r > 0, workspace=self.distill_ws)
        # rounded to bf16 by the product
        self.grad_table(r).copy_(torch.mm(self.dlogits.t(), h))
        dh = torch.mm(self.dlogits, self.table)
        if self.body is None:
            self.dhidden.copy_(dh)
        else:
            dhidden, *dwhole = torch.autograd.grad(out, [leaf, *kept], dh)
            self.dhidden.copy_(dhidden)
            for g, d in zip(self.rank_grads[r] if kept else (), dwhole):
                g.copy_(d)
        embed_grad(self.back, b.ids, self.dhidden, self.grad_table(r), self.embed_ws,
                   accumulate=True)

    def update(self, t: int, valid):
        """Reduce, clip and update every rank's shard."""
        spec = make_reduce(ZS_GRAD_F32 if self.f32_grads else ZS_GRAD_BF16, rank_tokens=valid)
        for k, s in enumerate(self.shards):
            ptrs = [self.grads[r].data_ptr() + s.shard_offset * self.grads.element_size()
                    for r in range(self.n_d)]
            shard_grad_reduce(s, spec, ptrs, self.mean[k], self.reduce_ws, self.sqnorm,
                              accumulate=k > 0)
        if self.whole:
            self._reduce_whole(valid)
        h = adamw(lr=self.lr, weight_decay=self.weight_decay, step=t,
                  max_grad_norm=self.max_grad_norm)
        for s, mean, (w, m, v) in zip(self.shards, self.mean, self.state):
            zero_shard_step(s, h, mean_in=mean, sqnorm=self.sqnorm, master=w, exp_avg=m,
                            exp_avg_sq=v, param_out=self.gather)

        if self.whole:
            w, m, v = self.whole_state
            # clipped already: no clip in the step
            plain = adamw(lr=self.lr, weight_decay=self.weight_decay, step=t)
            zero_shard_step(self.whole_shard, plain, mean_in=self.whole_mean, master=w, exp_avg=m,
                            exp_avg_sq=v, param_out=self.whole_gather)

    def _reduce_whole(self, valid):
        """The whole parameters' mean gradients; their norm into the shards', and
        the clipped gradients into the flat buffer of their step."""
        total = sum(valid)
        for k, g in enumerate(self.whole_grads):
            g.zero_()
            for r in range(self.n_d):
                g.add_(self.rank_grads[r][k].float(), alpha=valid[r] / total)
        tensors_sqnorm(self.whole_list, self.sqnorm, accumulate=True)
        if self.max_grad_norm > 0.0:
            tensors_clip(self.whole_list, self.max_grad_norm, self.sqnorm)
        else:                                   # no clip, as in zero_shard_step
            for flat, g in zip(self.whole_list.out, self.whole_grads):
                flat.copy_(g)

    def step(self, t: int, batches):
        """One optimizer step at bias-correction step t from one batch a rank."""
        for r, b in enumerate(batches):
            self.rank_pass(r, b)
        self.update(t, [b.valid for b in batches])
