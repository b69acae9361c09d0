"""Plain 64-bit forms of the position-bias calls (the oracle of their tests)."""
import math

import torch

U = 2.0 ** -24


def side_bucket(n, buckets, far):
    """The definition in whole numbers: E, plus the steps k whose border
    n^m >= E^(m-k) far^k is reached."""
    exact = buckets // 2
    if n < exact:
        return n
    m = buckets - exact
    return exact + sum(n ** m >= exact ** (m - k) * far ** k for k in range(1, m))


def bucket_table(r):
    """Buckets of distances 0..max_distance of one side."""
    side = r.buckets // 2 if r.bidirectional else r.buckets
    return side, torch.tensor([side_bucket(n, side, r.max_distance)
                               for n in range(r.max_distance + 1)])


def buckets_of(r, d):
    side, table = bucket_table(r)
    far = r.max_distance
    if r.bidirectional:
        return table[d.abs().clamp(max=far)] + side * (d > 0)
    return table[(-d).clamp(0, far)]


def positions(r, b, lengths, starts):
    """(distances, seen) of sequence b, [Q, K] on the CPU."""
    start = r.query_start if starts is None else int(starts[b])
    i = torch.arange(r.queries)[:, None] + start
    j = torch.arange(r.keys)[None, :]
    seen = torch.ones((r.queries, r.keys), dtype=torch.bool)
    if lengths is not None:
        seen &= j < int(lengths[b])
    if r.causal:
        seen &= j <= i
    return j - i, seen


def ref_bias(r, table, scores, lengths, starts):
    """(values, the sizes that fp32 roundings scale with), float64 [B, H, Q, K]."""
    out = torch.full((r.batch, r.heads, r.queries, r.keys), -math.inf, dtype=torch.float64)
    size = torch.zeros_like(out)
    table = table.cpu().double()
    scale = float(torch.tensor(r.scale, dtype=torch.float32))
    for b in range(r.batch):
        d, seen = positions(r, b, lengths, starts)
        bias = table[buckets_of(r, d)].permute(2, 0, 1)
        value = bias if scores is None else scores[b].cpu().double() * scale + bias
        out[b] = torch.where(seen, value, -math.inf)
        size[b] = torch.where(seen, value.abs(), 0.0)
    return out, size


def ref_grad(r, grad, lengths, starts):
    """(table gradient, sums of absolute values, scores' gradient), float64."""
    total = torch.zeros((r.buckets, r.heads), dtype=torch.float64)
    size = torch.zeros_like(total)
    scores = torch.zeros((r.batch, r.heads, r.queries, r.keys), dtype=torch.float64)
    scale = float(torch.tensor(r.scale, dtype=torch.float32))
    for b in range(r.batch):
        d, seen = positions(r, b, lengths, starts)
        u = buckets_of(r, d).reshape(-1)
        g = torch.where(seen, grad[b].cpu().double(), 0.0)
        flat = g.reshape(r.heads, -1).t()
        total.index_add_(0, u, flat)
        size.index_add_(0, u, flat.abs())
        scores[b] = g * scale
    return total, size, scores
