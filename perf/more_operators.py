"""Cases of the operators on many tensors (squared norm, clipping) and on the
position-bias table (bias by buckets of relative position, and its gradient).

``run`` computes a case either with elementary torch operations in 32 bits, 64
for long sums (``own`` false), or through the framework's entry points (``own``
true), on the same inputs.  ``exact`` gives the same outputs from the
definitions in 64 bits.
"""
from __future__ import annotations

import math
import random
from decimal import Decimal, localcontext

import torch

own = False

_BYTES = {"bf16": 2, "f32": 4}
_TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- the cases ---------------------------------------------------------------------

def _tensors(name, calls, shapes, count, lo=1, hi=1, types="f32", out="f32", limit=0.5,
             per_tensor=False, sizes_seed=0):
    """calls: "norm" (the squared norm alone), "clip" (by a norm that is there
    already), "pair" (the norm added to a shard's, then the clip) or "both" (one
    call).  out: the type of the flat buffer the clipped tensors go to, or
    "place".  limit: max_norm as a multiple of the global norm."""
    return {"name": name, "op": "tensors", "calls": calls, "shapes": shapes, "count": count,
            "lo": lo, "hi": hi, "types": types, "out": out, "limit": limit,
            "per_tensor": per_tensor, "sizes_seed": sizes_seed}


def _bias(name, op, batch, heads, queries, keys, dtype="bf16", table="f32", buckets=32,
          far=128, two_sided=True, causal=False, start=0, ragged=False, scores=False, scale=1.0):
    """op: "bias" or "bias_grad".  scores: the bias is added to scores (the
    gradient also leaves the scores').  ragged: a key length for each sequence
    (one token a sequence: its own position too)."""
    return {"name": name, "op": op, "batch": batch, "heads": heads, "queries": queries,
            "keys": keys, "dtype": dtype, "table": table, "buckets": buckets, "far": far,
            "two_sided": two_sided, "causal": causal, "start": start, "ragged": ragged,
            "scores": scores, "scale": scale}


def listed():
    return [
        # what is too small to shard in a small model: norm weights, biases and
        # a position table, kept whole on every rank; latency only
        _tensors("norm_small_set", "norm", "ragged", 26, 1, 4096),
        # the bf16 gradients of two FSDP units of 218,112,000 parameters, tensor
        # by tensor, each tensor's norm kept for the log
        _tensors("norm_two_units", "norm", "unit", 2, types="bf16", per_tensor=True),
        # a small block's gradients clipped into the fp32 buffer of the step,
        # by a norm that another pass has left
        _tensors("clip_small_block", "clip", "ragged", 16, 64, 262144, types="bf16"),
        # a sharded run: the norm is added to the shard's, other ranks' is added
        # in the clip; the largest: 872 million fp32 gradients
        _tensors("pair_four_units", "pair", "unit", 4),
        # many experts' tensors of both types and every size, flattened
        _tensors("both_ragged_1500", "both", "ragged", 1500, 1, 600000, types="mixed",
                 per_tensor=True, sizes_seed=1),
        # the ordinary step of a settled run: the norm is within the limit
        _tensors("both_within_limit", "both", "unit", 1, out="place", limit=2.0),
        # one token of a decoder against its cache: latency only
        _bias("bias_one_token", "bias", 1, 32, 1, 4099, two_sided=False, start=4098),
        # 64 sequences of different lengths, one token each: bias onto scores
        _bias("bias_decode_batch", "bias", 64, 16, 1, 8192, two_sided=False, ragged=True,
              scores=True, scale=0.125),
        # the dense bias of one layer at 4096 positions, for an attention call
        # that takes it
        _bias("bias_dense_4k", "bias", 1, 32, 4096, 4096),
        # an evaluation-sized batch
        _bias("grad_small", "bias_grad", 2, 8, 300, 300, dtype="f32"),
        # the second part of a causal sequence, odd sizes: both gradients
        _bias("grad_scores_odd", "bias_grad", 4, 12, 1023, 2051, two_sided=False, causal=True,
              start=1028, scores=True, scale=0.125),
        # a training micro-batch of padded sequences
        _bias("grad_padded_2k", "bias_grad", 8, 16, 2048, 2048, ragged=True),
    ]


def _spread(rng, lo, hi):
    """A size spread over the logarithm of [lo, hi], odd ones among them."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tensors", "bias", "bias_grad"])
    if op == "tensors":
        calls = rng.choice(["norm", "clip", "pair", "both"])
        limit = rng.choice([0.01, 0.5, 0.9, 2.0])
        # in place only where a second pass finds the same gradients
        out = rng.choice(["bf16", "f32", "place" if limit > 1.0 else "f32"])
        types = rng.choice(["bf16", "f32", "mixed"])
        if rng.random() < 0.2:
            return _tensors("", calls, "unit", rng.choice([1, 2, 3]), types=types, out=out,
                            limit=limit, per_tensor=rng.random() < 0.5)
        count = _spread(rng, 1, 3000)
        return _tensors("", calls, "ragged", count, 1,
                        _spread(rng, 64, min(1 << 25, 800_000_000 // count)), types=types,
                        out=out, limit=limit, per_tensor=rng.random() < 0.5,
                        sizes_seed=rng.randrange(1 << 30))
    two_sided = rng.random() < 0.6
    buckets = rng.choice([8, 16, 32, 32, 64, 128])
    far = rng.choice([2, 4, 5, 8]) * buckets
    heads = rng.randint(1, 48)
    dtype = rng.choice(["bf16", "f32"])
    queries = 1 if op == "bias" and rng.random() < 0.3 else _spread(rng, 2, 4096)
    batch = _spread(rng, 1, 64)
    keys = _spread(rng, 16, 16384)
    # no more elements than the dense case has
    while batch * heads * queries * keys > 32 * 4096 * 4096 // (2 if dtype == "f32" else 1):
        batch, queries, keys = max(1, batch // 2), -(-queries // 2), max(16, keys * 3 // 4)
    start = rng.choice([0, max(0, keys - queries)])
    return _bias("", op, batch, heads, queries, keys, dtype=dtype,
                 table=rng.choice(["bf16", "f32"]), buckets=buckets, far=far,
                 two_sided=two_sided, causal=not two_sided and rng.random() < 0.5, start=start,
                 ragged=rng.random() < 0.5, scores=rng.random() < 0.5,
                 scale=rng.choice([1.0, 0.125, 0.3]))


# ---- what a user's program has in hand before the call --------------------------------

def _sizes(case):
    if case["shapes"] == "unit":
        # four projections, three matrices of the feed-forward part, two norms:
        # 218,112,000 parameters of an FSDP unit
        unit = [(4096, 4096)] * 4 + [(4096, 12288)] * 3 + [(4096,)] * 2
        return unit * case["count"]
    rng = random.Random(case["sizes_seed"])
    return [(_spread(rng, case["lo"], case["hi"]),) for _ in range(case["count"])]


def _types(case):
    kinds = {"mixed": ("bf16", "f32", "bf16")}.get(case["types"], (case["types"],))
    return [kinds[k % len(kinds)] for k in range(len(_sizes(case)))]


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, std=1.0, dtype="f32"):
        x = torch.empty(shape, device="cuda", dtype=_TORCH[dtype])
        return x.normal_(0.0, std, generator=gen)

    if case["op"] == "tensors":
        sizes, types = _sizes(case), _types(case)
        numel = [math.prod(s) for s in sizes]
        room = {t: sum(-(-n // 64) * 64 for n, k in zip(numel, types) if k == t)
                for t in ("bf16", "f32")}
        pool = {t: normal(n, std=1e-3, dtype=t) for t, n in room.items()}
        used = dict.fromkeys(pool, 0)
        grads = []
        for shape, n, t in zip(sizes, numel, types):
            grads.append(pool[t][used[t]:used[t] + n].view(shape))
            used[t] += -(-n // 64) * 64
        # gradients of different layers differ in size
        for k, t in enumerate(("bf16", "f32")):
            mine = [g for g, kind in zip(grads, types) if kind == t]
            if mine:
                torch._foreach_mul_(mine, [2.0 ** ((i * 5 + k) % 7 - 3) for i in range(len(mine))])
        # the shard's part of the squared norm, or all of it where it is there already
        q = sum(n * 1e-6 * 4.0 for n in numel)
        return {"grads": grads, "shard": torch.full((1,), q, dtype=torch.float64, device="cuda"),
                "other": q if case["calls"] == "pair" else 0.0, "max_norm": _limit(case, q)}
    batch, queries, keys = case["batch"], case["queries"], case["keys"]
    x = {"lengths": None, "starts": None}
    if case["ragged"]:
        lengths = torch.randint(max(1, keys // 4), keys + 1, (batch,), generator=gen,
                                device="cuda")
        lengths[0] = keys
        if batch > 4:
            lengths[batch // 2] = 0          # a slot of the batch that is not in use
        x["lengths"] = lengths.int()
        if queries == 1:
            x["starts"] = (lengths - 1).clamp(min=0).int()
    shape = (batch, case["heads"], queries, keys)
    if case["op"] == "bias":
        x["table"] = normal(case["buckets"], case["heads"], std=0.5, dtype=case["table"])
        x["scores"] = normal(*shape, std=2.0 / case["scale"], dtype=case["dtype"]) \
            if case["scores"] else None
    else:
        x["grad"] = normal(*shape, std=1e-3, dtype=case["dtype"])
    return x


def _limit(case, q):
    """max_norm at `limit` times about the norm of these gradients, whose squares
    are 2^-6 to 2^6 times 1e-6, from tensor to tensor: 12.2e-6 on average, 3q."""
    norm = {"clip": math.sqrt(q), "pair": math.sqrt(5.0 * q)}.get(case["calls"],
                                                                   math.sqrt(3.0 * q))
    # within the limit must hold however the sizes fall
    return case["limit"] * norm * (8.0 if case["limit"] > 1.0 else 1.0)


def prepare(case, seed):
    x = _inputs(case, seed)
    state = {"case": case, "in": x}
    if not own:
        return state
    import fsdp_sharded_optimizer_zero_amd as Z
    kind = {"bf16": Z.ZS_BF16, "f32": Z.ZS_F32}
    if case["op"] == "tensors":
        grads = x["grads"]
        views = None
        if case["calls"] != "norm" and case["out"] != "place":
            numel = [g.numel() for g in grads]
            state["flat"] = torch.empty(sum(numel), dtype=_TORCH[case["out"]], device="cuda")
            views = [v.view(g.shape) for v, g in zip(state["flat"].split(numel), grads)]
        state["t"] = Z.make_tensors(grads, views)
        state["sqnorm"] = torch.zeros(1, dtype=torch.float64, device="cuda")
        state["each"] = torch.empty(len(grads), dtype=torch.float64, device="cuda") \
            if case["per_tensor"] and case["calls"] != "clip" else None
        return state
    r = Z.make_relpos(case["heads"], case["queries"], case["keys"], buckets=case["buckets"],
                      max_distance=case["far"], batch=case["batch"],
                      bidirectional=case["two_sided"], causal=case["causal"],
                      query_start=case["start"], scale=case["scale"], dtype=kind[case["dtype"]],
                      table_dtype=kind[case["table"]], id_dtype=Z.ZS_ID_I32)
    state["r"] = r
    shape = (case["batch"], case["heads"], case["queries"], case["keys"])
    if case["op"] == "bias":
        state["out"] = torch.empty(shape, dtype=_TORCH[case["dtype"]], device="cuda")
    else:
        state["dtable"] = torch.empty((case["buckets"], case["heads"]),
                                      dtype=_TORCH[case["table"]], device="cuda")
        state["dscores"] = torch.empty_like(x["grad"]) if case["scores"] else None
        state["ws"] = torch.empty(max(Z.zs_relpos_workspace_bytes(r), 16), dtype=torch.uint8,
                                  device="cuda")
    return state


# ---- one pass ----------------------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    if case["op"] == "tensors":
        return _plain_tensors(case, state["in"])
    if case["op"] == "bias":
        return _plain_bias(case, state["in"])
    return _plain_bias_grad(case, state["in"])


def _run_own(case, st):
    import fsdp_sharded_optimizer_zero_amd as Z
    x = st["in"]
    if case["op"] == "bias":
        Z.relpos_bias(st["r"], x["table"], st["out"], scores=x["scores"],
                      key_lengths=x["lengths"], query_starts=x["starts"])
        return {"out": st["out"]}
    if case["op"] == "bias_grad":
        Z.relpos_bias_grad(st["r"], x["grad"], st["dtable"], st["ws"], grad_scores=st["dscores"],
                           key_lengths=x["lengths"], query_starts=x["starts"])
        out = {"table": st["dtable"]}
        if case["scores"]:
            out["scores"] = st["dscores"]
        return out
    out = {}
    if case["calls"] == "clip":
        Z.tensors_clip(st["t"], x["max_norm"], x["shard"])
    elif case["calls"] == "pair":
        # the shard's pass left its squared norm in the scalar that is added to
        st["sqnorm"].copy_(x["shard"])
        Z.tensors_sqnorm(st["t"], st["sqnorm"], tensor_sqnorms=st["each"], accumulate=True)
        Z.tensors_clip(st["t"], x["max_norm"], st["sqnorm"], other_sqnorm=x["other"])
    elif case["calls"] == "both":
        Z.tensors_clip_norm(st["t"], x["max_norm"], st["sqnorm"], tensor_sqnorms=st["each"])
    else:
        Z.tensors_sqnorm(st["t"], st["sqnorm"], tensor_sqnorms=st["each"])
    if case["calls"] != "clip":
        out["sqnorm"] = st["sqnorm"]
        if st["each"] is not None:
            out["each"] = st["each"]
    if case["calls"] != "norm":
        out["clipped"] = x["grads"] if case["out"] == "place" else st["flat"]
    return out


# ---- the plain form ------------------------------------------------------------------------

def _plain_tensors(case, x):
    out = {}
    q = x["shard"]
    if case["calls"] != "clip":
        each = torch.stack([g.reshape(-1).double().square().sum() for g in x["grads"]])
        q = each.sum().reshape(1)
        if case["calls"] == "pair":
            q = q + x["shard"]
        out["sqnorm"] = q
        if case["per_tensor"]:
            out["each"] = each
    if case["calls"] != "norm":
        coef = (x["max_norm"] / (torch.sqrt(q + x["other"]) + 1e-6)).clamp(max=1.0).float()
        if case["out"] == "place":
            out["clipped"] = [(g.float() * coef).to(g.dtype) for g in x["grads"]]
        else:
            out["clipped"] = torch.cat([(g.reshape(-1).float() * coef).to(_TORCH[case["out"]])
                                        for g in x["grads"]])
    return out


def _edges(case):
    """(half, exact, the smallest distance of each bucket after the first
    logarithmic one), in whole numbers."""
    half = case["buckets"] // 2 if case["two_sided"] else case["buckets"]
    exact = half // 2
    m = half - exact
    edges = []
    for k in range(1, m):
        lo, hi = exact, case["far"]
        while lo < hi:
            n = (lo + hi) // 2
            if n ** m >= exact ** (m - k) * case["far"] ** k:
                hi = n
            else:
                lo = n + 1
        edges.append(lo)
    return half, exact, edges


def _plain_buckets(case, d):
    half, exact, edges = _edges(case)
    n = d.abs() if case["two_sided"] else (-d).clamp(min=0)
    steps = torch.bucketize(n, torch.tensor(edges, device=d.device), right=True)
    bucket = torch.where(n < exact, n, exact + steps)
    return bucket + half * (d > 0) if case["two_sided"] else bucket


def _positions(case, x, b):
    """(distances key - query of a sequence, which places it sees), [Q, K]."""
    start = case["start"] if x["starts"] is None else x["starts"][b].long()
    i = torch.arange(case["queries"], device="cuda")[:, None] + start
    j = torch.arange(case["keys"], device="cuda")[None, :]
    seen = torch.ones((case["queries"], case["keys"]), dtype=torch.bool, device="cuda")
    if x["lengths"] is not None:
        seen = seen & (j < x["lengths"][b])
    if case["causal"]:
        seen = seen & (j <= i)
    return j - i, seen


def _plain_bias(case, x):
    out = torch.empty((case["batch"], case["heads"], case["queries"], case["keys"]),
                      dtype=_TORCH[case["dtype"]], device="cuda")
    bias = None
    for b in range(case["batch"]):
        if bias is None or x["starts"] is not None or x["lengths"] is not None:
            d, seen = _positions(case, x, b)
        if bias is None or x["starts"] is not None:
            # rows of the table by bucket, heads first
            bias = x["table"].float()[_plain_buckets(case, d)].permute(2, 0, 1)
        value = bias if x["scores"] is None else x["scores"][b].float() * case["scale"] + bias
        out[b] = torch.where(seen, value, -math.inf)
    return {"out": out}


def _plain_bias_grad(case, x):
    queries, keys, heads = case["queries"], case["keys"], case["heads"]
    out = {}
    total = torch.zeros((heads, queries, keys), device="cuda")
    for b in range(case["batch"]):
        if b == 0 or x["lengths"] is not None:
            _, seen = _positions(case, x, b)
        g = torch.where(seen, x["grad"][b].float(), 0.0)
        total += g
        if case["scores"]:
            if b == 0:
                out["scores"] = torch.empty_like(x["grad"])
            out["scores"][b] = g * case["scale"]
    # sums along the diagonals: a row of keys + queries elements read as one of
    # keys + queries - 1 moves one place to the right in each next row
    wide = torch.cat([total.flip(1), torch.zeros((heads, queries, queries), device="cuda")], 2)
    flat = wide.reshape(heads, -1)[:, :queries * (keys + queries - 1)]
    diagonals = flat.view(heads, queries, keys + queries - 1).double().sum(1)
    d = torch.arange(keys + queries - 1, device="cuda") - (queries - 1) - case["start"]
    table = torch.zeros((case["buckets"], heads), dtype=torch.float64, device="cuda")
    table.index_add_(0, _plain_buckets(case, d), diagonals.t().contiguous())
    out["table"] = table.to(_TORCH[case["table"]])
    return out


# ---- from the definitions, in 64 bits --------------------------------------------------------

def exact(case, seed):
    x = _inputs(case, seed)
    if case["op"] == "tensors":
        return _exact_tensors(case, x)
    return _exact_bias(case, x) if case["op"] == "bias" else _exact_bias_grad(case, x)


def _exact_tensors(case, x):
    out = {}
    norms = [torch.linalg.vector_norm(g, dtype=torch.float64).item() for g in x["grads"]]
    q = float(x["shard"].item())
    if case["calls"] != "clip":
        own_q = math.fsum(n * n for n in norms)
        q = own_q + q if case["calls"] == "pair" else own_q
        out["sqnorm"] = torch.tensor([q], dtype=torch.float64, device="cuda")
        if case["per_tensor"]:
            out["each"] = torch.tensor([n * n for n in norms], dtype=torch.float64, device="cuda")
    if case["calls"] != "norm":
        coef = min(1.0, x["max_norm"] / (math.sqrt(q + x["other"]) + 1e-6))
        if case["out"] == "place":
            out["clipped"] = [g.double() * coef for g in x["grads"]]
        else:
            flat = torch.empty(sum(g.numel() for g in x["grads"]), dtype=torch.float64,
                               device="cuda")
            at = 0
            for g in x["grads"]:
                torch.mul(g.reshape(-1).double(), coef, out=flat[at:at + g.numel()])
                at += g.numel()
            out["clipped"] = flat
    return out


def _exact_buckets(case):
    """Bucket of every distance below `far`, from the logarithms in 60 digits."""
    half = case["buckets"] // 2 if case["two_sided"] else case["buckets"]
    linear = half // 2
    table = list(range(linear))
    with localcontext() as ctx:
        ctx.prec = 60
        ratio = (Decimal(case["far"]) / linear).ln()
        for n in range(linear, case["far"] + 1):
            step = (Decimal(n) / linear).ln() / ratio * (half - linear)
            # a whole number comes out within 1e-50 of itself
            table.append(min(half - 1, linear + int(step + Decimal("1e-40"))))
    return half, torch.tensor(table, device="cuda")


def _exact_lookup(case, half, table, d):
    if case["two_sided"]:
        return table[d.abs().clamp(max=case["far"])] + torch.where(d > 0, half, 0)
    return table[(-d).clamp(min=0, max=case["far"])]


def _exact_bias(case, x):
    half, table = _exact_buckets(case)
    out = torch.full((case["batch"], case["heads"], case["queries"], case["keys"]), -math.inf,
                     dtype=torch.float64, device="cuda")
    weights = x["table"].double()
    for b in range(case["batch"]):
        d, seen = _positions(case, x, b)
        bucket = _exact_lookup(case, half, table, d)
        for h in range(case["heads"]):
            value = weights[:, h][bucket]
            if x["scores"] is not None:
                value = torch.addcmul(value, x["scores"][b, h].double(),
                                      torch.full_like(value, case["scale"]))
            out[b, h][seen] = value[seen]
    return {"out": out}


def _exact_bias_grad(case, x):
    half, table = _exact_buckets(case)
    out = {"table": torch.zeros((case["buckets"], case["heads"]), dtype=torch.float64,
                                device="cuda")}
    if case["scores"]:
        out["scores"] = torch.zeros_like(x["grad"], dtype=torch.float64)
    for b in range(case["batch"]):
        d, seen = _positions(case, x, b)
        bucket = _exact_lookup(case, half, table, d)[seen]
        for h in range(case["heads"]):
            g = x["grad"][b, h].double()[seen]
            out["table"][:, h] += torch.bincount(bucket, weights=g, minlength=case["buckets"])
            if case["scores"]:
                out["scores"][b, h][seen] = g * case["scale"]
    return out


# ---- what one pass cannot do without ---------------------------------------------------------

def _seen(case):
    """Places that are seen, expected over the lengths that are drawn."""
    share = 1.0
    if case["ragged"] and case["batch"] > 1:
        some = case["batch"] - 1 - (1 if case["batch"] > 4 else 0)
        share = (1.0 + 0.625 * some) / case["batch"]
    places = float(case["queries"]) * case["keys"]
    if case["causal"]:
        start = case["start"]
        places = float(sum(max(0, min(case["keys"], i + start + 1))
                           for i in range(case["queries"])))
    return places * share * case["batch"] * case["heads"]


def work(case):
    if case["op"] == "tensors":
        numel = [math.prod(s) for s in _sizes(case)]
        read = sum(n * _BYTES[t] for n, t in zip(numel, _types(case)))
        wrote = 0
        if case["calls"] != "norm":
            # in place and within the limit, the gradients stay as they are
            wrote = 0 if case["out"] == "place" else sum(numel) * _BYTES[case["out"]]
        if case["calls"] == "clip" and case["out"] == "place":
            read = 0
        flops = {"norm": 2, "clip": 1}.get(case["calls"], 3)
        return {"bytes": read + wrote + 8, "flops": flops * sum(numel)}
    size, seen = _BYTES[case["dtype"]], _seen(case)
    places = case["batch"] * case["heads"] * case["queries"] * case["keys"]
    small = case["buckets"] * case["heads"] * _BYTES[case["table"]]
    if case["op"] == "bias":
        return {"bytes": size * (places + (seen if case["scores"] else 0)) + small,
                "flops": 2 * seen}
    return {"bytes": size * (seen + (places if case["scores"] else 0)) + small,
            "flops": 2 * seen}
