"""Cases of the vocabulary-table operators: embedding lookup and gradient, and
distillation from a teacher's top logits.

``run`` computes a case either with elementary torch operations in 32 bits
(``own`` false) or through the framework's entry points (``own`` true), on the
same inputs.  ``exact`` gives the same outputs from the definitions in 64 bits.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_BYTES = {"bf16": 2, "f32": 4, "i32": 4, "i64": 8}
_TORCH = {"bf16": torch.bfloat16, "f32": torch.float32, "i32": torch.int32, "i64": torch.int64}


# ---- the cases ---------------------------------------------------------------------

def _lookup(name, tokens, rows, dim, vocab=None, first=0, table="bf16", act="bf16", ids="i64",
            scale=1.0):
    return {"name": name, "op": "lookup", "tokens": tokens, "rows": rows, "dim": dim,
            "vocab": vocab or rows, "first": first, "table": table, "act": act, "ids": ids,
            "scale": scale}


def _grad(name, tokens, rows, dim, vocab=None, first=0, table="f32", act="bf16", ids="i64",
          scale=1.0, micro=1):
    return {"name": name, "op": "grad", "tokens": tokens, "rows": rows, "dim": dim,
            "vocab": vocab or rows, "first": first, "table": table, "act": act, "ids": ids,
            "scale": scale, "micro": micro}


def _distill(name, calls, rows, vocab, k, logits="bf16", teacher="f32", ids="i32", tau=1.0,
             alpha=1.0, labels=True, mass=False):
    return {"name": name, "op": "distill", "calls": calls, "rows": rows, "vocab": vocab, "k": k,
            "logits": logits, "teacher": teacher, "ids": ids, "tau": tau, "alpha": alpha,
            "labels": labels, "mass": mass}


def listed():
    return [
        # one token of a step-by-step evaluation during training: latency only
        _lookup("lookup_one_token", 1, 32000, 4096),
        # a micro-batch of four 4096-token sequences, the table scaled by sqrt(dim)
        _lookup("lookup_microbatch", 16384, 128256, 4096, ids="i32", scale=64.0),
        # one of eight row ranges of a table, from the fp32 master, odd width:
        # most ids belong to other ranges
        _lookup("lookup_row_range_odd", 2051, 6283, 771, vocab=50257, first=6283, table="f32"),
        # a byte-level table and a few tokens: latency only
        _grad("grad_byte_table", 37, 259, 768),
        # a GPT-2-small-sized table, gradient in bf16, one 4096-token sequence
        _grad("grad_4k_bf16", 4096, 50257, 768, table="bf16", ids="i32"),
        # gradient accumulation: the first micro-batch sets, the second adds
        _grad("grad_two_microbatches", 8192, 128256, 4096, micro=2, scale=64.0),
        # one row range of a table, odd width, fp32 activations
        _grad("grad_row_range_odd", 5003, 6283, 771, vocab=50257, first=0, act="f32"),
        # the largest: 65536 tokens into the bf16 gradient of a 128256-row table
        _grad("grad_64k_bf16", 65536, 128256, 4096, table="bf16"),
        # loss and gradient as two calls (autograd order), a few short
        # sequences, odd vocabulary (rows not vector-aligned)
        _distill("pair_few_rows_odd", "pair", 64, 50257, 16),
        # the same calls on a micro-batch: fp32 logits, mixed with the labels,
        # teacher probabilities from the full distribution
        _distill("pair_f32", "pair", 2048, 50257, 50, logits="f32", ids="i64", tau=2.0,
                 alpha=0.5, mass=True),
        # loss and gradient of few rows in one call: each row spread over the GPU
        _distill("step_few_rows", "step", 24, 128256, 128, tau=1.5, alpha=0.7),
        # a training micro-batch in one call: padded rows, temperature 2
        _distill("step_8k_rows", "step", 8192, 128256, 64, teacher="bf16", tau=2.0),
    ]


def _spread(rng, lo, hi):
    """A size spread over the logarithm of [lo, hi], odd ones among them."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["lookup", "grad", "distill"])
    if op == "distill":
        vocab = _spread(rng, 300, 160000)
        rows = _spread(rng, 1, max(2, min(8192, 8192 * 128256 // (4 * vocab))))
        alpha = rng.choice([1.0, 0.9, 0.5])
        return _distill("", rng.choice(["pair", "step"]), rows, vocab,
                        _spread(rng, 1, 256), logits=rng.choice(["bf16", "f32"]),
                        teacher=rng.choice(["bf16", "f32"]), ids=rng.choice(["i32", "i64"]),
                        tau=rng.choice([1.0, 1.0, 1.5, 2.0, 4.0]), alpha=alpha,
                        labels=alpha < 1.0 or rng.random() < 0.7, mass=rng.random() < 0.5)
    vocab = _spread(rng, 256, 160000)
    dim = _spread(rng, 64, 8192)
    if rng.random() < 0.6:
        dim = max(64, dim // 64 * 64)
    rows, first = vocab, 0
    if rng.random() < 0.4:
        parts = rng.choice([2, 4, 8])
        rows = -(-vocab // parts)
        first = rows * rng.randrange(parts)
        rows = max(1, min(rows, vocab - first))
    scale = rng.choice([1.0, round(math.sqrt(dim), 3)])
    ids = rng.choice(["i32", "i64"])
    if op == "lookup":
        tokens = _spread(rng, 1, 65536)
        return _lookup("", tokens, rows, dim, vocab, first, table=rng.choice(["bf16", "f32"]),
                       act=rng.choice(["bf16", "f32"]), ids=ids, scale=scale)
    # no more than the largest listed gradient: its table and its tokens
    dim = max(1, min(dim, 128256 * 4096 // (3 * rows)))
    tokens = _spread(rng, 1, min(65536, 65536 * 4096 // (4 * dim)))
    return _grad("", tokens, rows, dim, vocab, first, table=rng.choice(["bf16", "f32"]),
                 act=rng.choice(["bf16", "f32"]), ids=ids, scale=scale, micro=rng.choice([1, 2]))


# ---- what a user's program has in hand before the call --------------------------------

def _token_ids(case, gen):
    """Token ids as a vocabulary ordered by frequency gives them (the density
    of id v falls as 1/v), a run of padding (-1) at the end of the batch."""
    n, vocab = case["tokens"], case["vocab"]
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    ids = (torch.exp(u * math.log(vocab + 1.0)) - 1.0).long().clamp_(0, vocab - 1)
    if n >= 16:
        ids[n - n // 16:] = -1
    # whatever the row range, a token names one of its rows
    ids[0] = case["first"] + int(torch.randint(0, case["rows"], (1,), generator=gen,
                                               device="cuda"))
    return ids.to(_TORCH[case["ids"]])


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, std=1.0, dtype="f32"):
        x = torch.empty(shape, device="cuda", dtype=_TORCH[dtype])
        return x.normal_(0.0, std, generator=gen)

    if case["op"] == "lookup":
        return {"ids": _token_ids(case, gen),
                "table": normal(case["rows"], case["dim"], std=0.02, dtype=case["table"])}
    if case["op"] == "grad":
        return {"ids": [_token_ids(case, gen) for _ in range(case["micro"])],
                "act": [normal(case["tokens"], case["dim"], std=1e-3, dtype=case["act"])
                        for _ in range(case["micro"])]}
    n, vocab, k = case["rows"], case["vocab"], min(case["k"], case["vocab"])
    logits = normal(n, vocab, std=2.0, dtype=case["logits"])
    # the teacher's entries: distinct ids, values falling from about 12; the
    # student roughly agrees, some rows offer fewer entries (id -1)
    start = torch.randint(0, vocab, (n, 1), generator=gen, device="cuda")
    step = max(1, vocab // k)
    ids = (start + step * torch.arange(k, device="cuda")) % vocab
    value = 12.0 - 0.25 * torch.arange(k, device="cuda") + normal(n, k, std=0.3)
    value = value.sort(dim=1, descending=True).values
    student = (value + normal(n, k, std=1.0)).to(logits.dtype)
    logits.scatter_(1, ids, student)
    short = torch.rand(n, generator=gen, device="cuda") < 0.1
    keep = torch.arange(k, device="cuda")[None, :] < torch.where(short, (k + 1) // 2, k)[:, None]
    tau = case["tau"]
    # log of the mass of the teacher's full distribution: its entries hold most of it
    lse = torch.logsumexp(torch.where(keep, value, -math.inf) / tau, dim=1) + 0.05
    # the label is mostly one of the teacher's entries
    pick = torch.randint(0, k, (n, 1), generator=gen, device="cuda")
    label = torch.gather(ids, 1, pick)[:, 0]
    if n >= 8:
        label[n - n // 8:] = -100          # padded positions
    return {"logits": logits,
            "teacher_ids": torch.where(keep, ids, -1).to(_TORCH[case["ids"]]),
            "teacher_logits": value.to(_TORCH[case["teacher"]]),
            "teacher_lse": lse if case["mass"] else None,
            "labels": label.to(_TORCH[case["ids"]]) if case["labels"] else None}


def _distill_scale(case):
    """1 / the rows that count, as a program that makes the labels knows them."""
    n = case["rows"]
    return 1.0 / (n - n // 8 if case["labels"] and n >= 8 else n)


def prepare(case, seed):
    state = {"case": case, "in": _inputs(case, seed)}
    if own:
        import fsdp_sharded_optimizer_zero_amd as Z
        kind = {"bf16": Z.ZS_BF16, "f32": Z.ZS_F32, "i32": Z.ZS_ID_I32, "i64": Z.ZS_ID_I64}

        def buffer(shape, dtype):
            return torch.empty(shape, dtype=dtype, device="cuda")

        def workspace(nbytes):
            return buffer(max(nbytes, 16), torch.uint8)

        if case["op"] in ("lookup", "grad"):
            e = Z.make_embed(case["tokens"], case["rows"], case["dim"], first_row=case["first"],
                             id_dtype=kind[case["ids"]], table_dtype=kind[case["table"]],
                             act_dtype=kind[case["act"]], scale=case["scale"])
            state["e"] = e
            if case["op"] == "lookup":
                state["out"] = buffer((case["tokens"], case["dim"]), _TORCH[case["act"]])
            else:
                state["out"] = buffer((case["rows"], case["dim"]), _TORCH[case["table"]])
                state["ws"] = workspace(Z.zs_embed_workspace_bytes(e))
        else:
            n, vocab = case["rows"], case["vocab"]
            d = Z.make_distill(n, vocab, min(case["k"], vocab), logits_dtype=kind[case["logits"]],
                               teacher_dtype=kind[case["teacher"]], id_dtype=kind[case["ids"]],
                               temperature=case["tau"], alpha=case["alpha"],
                               scale=_distill_scale(case))
            state["d"] = d
            state["ws"] = workspace(Z.zs_distill_workspace_bytes(d))
            state["loss"] = buffer((n,), torch.float32)
            state["lse"] = buffer((n, 2), torch.float32)
            state["loss_sum"] = buffer((1,), torch.float32)
            state["counted"] = buffer((1,), torch.int64)
            state["grad"] = buffer((n, vocab), _TORCH[case["logits"]])
    return state


# ---- one pass ----------------------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    if case["op"] == "lookup":
        return _plain_lookup(case, state["in"])
    if case["op"] == "grad":
        return _plain_grad(case, state["in"])
    return _plain_distill(case, state["in"])


def _run_own(case, st):
    import fsdp_sharded_optimizer_zero_amd as Z
    x = st["in"]
    if case["op"] == "lookup":
        Z.embed_lookup(st["e"], x["ids"], x["table"], st["out"])
        return st["out"]
    if case["op"] == "grad":
        for j in range(case["micro"]):
            Z.embed_grad(st["e"], x["ids"][j], x["act"][j], st["out"], st["ws"],
                         accumulate=j > 0)
        return st["out"]
    targets = dict(teacher_lse=x["teacher_lse"], labels=x["labels"])
    sums = dict(loss_sum=st["loss_sum"], counted=st["counted"], workspace=st["ws"])
    out = {name: st[name] for name in ("loss", "loss_sum", "counted", "grad")}
    if case["calls"] == "step":
        Z.distill_loss_grad(st["d"], x["logits"], x["teacher_ids"], x["teacher_logits"],
                            st["loss"], st["grad"], **sums, **targets)
        return out
    Z.distill_loss(st["d"], x["logits"], x["teacher_ids"], x["teacher_logits"], st["loss"],
                   st["lse"], **sums, **targets)
    Z.distill_grad(st["d"], x["logits"], x["teacher_ids"], x["teacher_logits"], st["lse"],
                   st["grad"], **targets)
    out["lse"] = st["lse"]
    return out


# ---- the plain form ------------------------------------------------------------------------

def _plain_lookup(case, x):
    row = x["ids"].long() - case["first"]
    here = (row >= 0) & (row < case["rows"])
    out = x["table"][row.clamp(0, case["rows"] - 1)].float() * case["scale"]
    out = torch.where(here[:, None], out, 0.0)
    return out.to(_TORCH[case["act"]])


def _plain_grad(case, x):
    grad = None
    for ids, act in zip(x["ids"], x["act"]):
        row = ids.long() - case["first"]
        here = (row >= 0) & (row < case["rows"])
        total = torch.zeros((case["rows"], case["dim"]), device="cuda")
        total.index_add_(0, row.clamp(0, case["rows"] - 1),
                         torch.where(here[:, None], act.float(), 0.0))
        total *= case["scale"]
        grad = (total if grad is None else grad.float() + total).to(_TORCH[case["table"]])
    return grad


def _plain_distill(case, x):
    tau, alpha, vocab = case["tau"], case["alpha"], case["vocab"]
    s = x["logits"].float()
    ids = x["teacher_ids"].long()
    value = x["teacher_logits"].float()
    there = (ids >= 0) & (ids < vocab) & (value > -math.inf)
    at = ids.clamp(0, vocab - 1)
    u = torch.where(there, value, -math.inf) / tau
    if x["teacher_lse"] is None:
        top = u.amax(dim=1, keepdim=True).clamp(min=-3e38)
        w = torch.exp(u - top)
        total = w.sum(dim=1, keepdim=True)
        p = torch.where(total > 0, w / total, 0.0)
        logp = u - top - torch.log(total)
    else:
        logp = u - x["teacher_lse"][:, None]
        p = torch.exp(logp)
    counts = there.any(dim=1) if alpha == 1.0 else torch.ones_like(there[:, 0])
    if x["labels"] is not None:
        label = x["labels"].long()
        counts &= (label >= 0) & (label < vocab)
        label = label.clamp(0, vocab - 1)[:, None]

    def log_sum_exp(z):
        m = z.amax(dim=1, keepdim=True)
        return m + torch.log(torch.exp(z - m).sum(dim=1, keepdim=True))

    z = s / tau
    lse = log_sum_exp(z)
    logq = torch.gather(z, 1, at) - lse
    kd = torch.where(p > 0, p * (logp - logq), 0.0).sum(dim=1)
    loss = alpha * tau * tau * kd
    lse1 = torch.zeros_like(lse)
    if alpha < 1.0:
        lse1 = log_sum_exp(s)
        loss = loss + (1.0 - alpha) * (lse1 - torch.gather(s, 1, label))[:, 0]
    loss = torch.where(counts, loss, 0.0)
    out = {"loss": loss, "loss_sum": loss.double().sum().float().reshape(1),
           "counted": counts.sum().reshape(1)}
    if case["calls"] == "pair":
        out["lse"] = torch.where(counts[:, None], torch.cat([lse, lse1], dim=1), 0.0)
    grad = torch.exp(z - lse) * (alpha * tau * p.sum(dim=1, keepdim=True))
    grad.scatter_add_(1, at, -alpha * tau * torch.where(there, p, 0.0))
    if alpha < 1.0:
        grad += (1.0 - alpha) * torch.exp(s - lse1)
        grad.scatter_add_(1, label, torch.full_like(lse, alpha - 1.0))
    grad = torch.where(counts[:, None], grad * _distill_scale(case), 0.0)
    out["grad"] = grad.to(x["logits"].dtype)
    return out


# ---- from the definitions, in 64 bits --------------------------------------------------------

def exact(case, seed):
    x = _inputs(case, seed)
    if case["op"] == "lookup":
        out = torch.zeros((case["tokens"], case["dim"]), dtype=torch.float64, device="cuda")
        local = x["ids"].to(torch.int64) - case["first"]
        t = torch.nonzero((local >= 0) & (local < case["rows"]))[:, 0]
        out[t] = x["table"].double()[local[t]] * case["scale"]
        return out
    if case["op"] == "grad":
        grad = torch.zeros((case["rows"], case["dim"]), dtype=torch.float64, device="cuda")
        for ids, act in zip(x["ids"], x["act"]):
            local = ids.to(torch.int64) - case["first"]
            t = torch.nonzero((local >= 0) & (local < case["rows"]))[:, 0]
            grad.index_put_((local[t],), act[t].double() * case["scale"], accumulate=True)
        return grad
    n, vocab = case["rows"], case["vocab"]
    loss = torch.zeros(n, dtype=torch.float64, device="cuda")
    lse = torch.zeros((n, 2), dtype=torch.float64, device="cuda")
    counts = torch.zeros(n, dtype=torch.float64, device="cuda")
    grad = torch.zeros((n, vocab), dtype=torch.float64, device="cuda")
    for a in range(0, n, 512):
        _exact_rows(case, x, a, min(n, a + 512), loss, lse, counts, grad)
    out = {"loss": loss, "loss_sum": loss.sum().reshape(1),
           "counted": counts.sum().long().reshape(1), "grad": grad}
    if case["calls"] == "pair":
        out["lse"] = lse
    return out


def _exact_rows(case, x, a, b, loss, lse, counts, grad):
    """Rows [a, b) with a softmax over the whole vocabulary and the teacher
    laid out dense over it."""
    tau, alpha, vocab = case["tau"], case["alpha"], case["vocab"]
    s = x["logits"][a:b].double()
    ids, u = x["teacher_ids"][a:b].long(), x["teacher_logits"][a:b].double() / tau
    there = (ids >= 0) & (ids < vocab) & torch.isfinite(u)
    if x["teacher_lse"] is None:
        norm = torch.logsumexp(u.masked_fill(~there, -math.inf), dim=1, keepdim=True)
    else:
        norm = x["teacher_lse"][a:b, None].double()
    p = torch.exp(u - norm).masked_fill(~there, 0.0)
    dense = torch.zeros_like(s).scatter_add_(1, ids.masked_fill(~there, 0), p)
    mass = p.sum(dim=1, keepdim=True)
    entropy = torch.xlogy(p, p).sum(dim=1)
    logq = torch.log_softmax(s / tau, dim=1)
    value = alpha * tau * tau * (entropy - (dense * logq).sum(dim=1))
    slope = alpha * tau * (mass * logq.exp() - dense)
    ok = there.any(dim=1) if alpha == 1.0 else torch.ones_like(there[:, 0])
    if x["labels"] is not None:
        label = x["labels"][a:b].long()
        ok = ok & (label >= 0) & (label < vocab)
        if alpha < 1.0:
            logq1 = torch.log_softmax(s, dim=1)
            hit = torch.zeros_like(s).scatter_(1, label.clamp(0, vocab - 1)[:, None], 1.0)
            value = value - (1.0 - alpha) * (hit * logq1).sum(dim=1)
            slope = slope + (1.0 - alpha) * (logq1.exp() - hit)
    loss[a:b] = value.masked_fill(~ok, 0.0)
    lse[a:b, 0] = torch.logsumexp(s / tau, dim=1).masked_fill(~ok, 0.0)
    if alpha < 1.0:
        lse[a:b, 1] = torch.logsumexp(s, dim=1).masked_fill(~ok, 0.0)
    counts[a:b] = ok.double()
    grad[a:b] = (slope * _distill_scale(case)).masked_fill(~ok[:, None], 0.0)


# ---- what one pass cannot do without ---------------------------------------------------------

def _touched(case):
    """(tokens whose id lies in the row range, distinct rows they name), expected."""
    n, vocab = case["tokens"], case["vocab"]
    n -= n // 16 if n >= 16 else 0
    v = np.arange(case["first"], case["first"] + case["rows"], dtype=np.float64)
    p = np.log((v + 2.0) / (v + 1.0)) / math.log(vocab + 1.0)
    return n * float(p.sum()), float((1.0 - (1.0 - p) ** n).sum())


def work(case):
    if case["op"] == "lookup":
        _, distinct = _touched(case)
        n, dim = case["tokens"], case["dim"]
        return {"bytes": n * _BYTES[case["ids"]] + distinct * dim * _BYTES[case["table"]]
                + n * dim * _BYTES[case["act"]], "flops": n * dim}
    if case["op"] == "grad":
        here, distinct = _touched(case)
        dim, g = case["dim"], _BYTES[case["table"]]
        per = case["tokens"] * _BYTES[case["ids"]] + here * dim * _BYTES[case["act"]]
        return {"bytes": case["micro"] * per + case["rows"] * dim * g
                + (case["micro"] - 1) * 2 * distinct * dim * g,
                "flops": case["micro"] * here * dim}
    n, vocab, k = case["rows"], case["vocab"], min(case["k"], case["vocab"])
    counted = n - n // 8 if case["labels"] and n >= 8 else n
    size = _BYTES[case["logits"]]
    reads = {"pair": 2, "step": 1}[case["calls"]]
    exps = 2 * (1 if case["alpha"] == 1.0 else 2)
    return {"bytes": (reads * counted + n) * vocab * size
            + counted * k * (_BYTES[case["ids"]] + _BYTES[case["teacher"]]),
            "flops": 4 * exps * counted * vocab}
