"""Plain 64-bit forms of the vocabulary-table operators (the oracle of their
tests), the error bounds the tests allow, and buffers with guards.

u = 2^-24 is the largest relative error of one fp32 rounding; half a step of
the output type is torch.finfo(t).eps / 2.
"""
import math

import torch

import fsdp_sharded_optimizer_zero_amd as Z

U = 2.0 ** -24
KIND = {torch.bfloat16: Z.ZS_BF16, torch.float32: Z.ZS_F32, torch.int32: Z.ZS_ID_I32,
        torch.int64: Z.ZS_ID_I64}
GUARD = 37


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def guarded(rows, width, pitch, dtype, fill=-7.0, device="cuda"):
    """A flat buffer of `rows` rows, `pitch` apart, all of it `fill`, with
    GUARD elements behind; (buffer, view of the rows)."""
    n = (rows - 1) * pitch + width if rows else 0
    buf = torch.full((n + GUARD,), fill, dtype=dtype, device=device)
    return buf, buf[:n].as_strided((rows, width), (pitch, 1))


def assert_guards(buf, rows, width, pitch, fill=-7.0):
    """Only the rows' own columns may differ from `fill`."""
    mask = torch.ones_like(buf, dtype=torch.bool)
    if rows:
        mask[:(rows - 1) * pitch + width].as_strided((rows, width), (pitch, 1)).fill_(False)
    assert bool((buf[mask] == fill).all()), "written outside the rows"


# ---- embedding ---------------------------------------------------------------------

def ref_lookup(ids, table, first, scale):
    row = ids.cpu().long() - first
    table = table.cpu().double()
    here = (row >= 0) & (row < table.shape[0])
    out = table[row.clamp(0, table.shape[0] - 1)] * scale
    return torch.where(here[:, None], out, 0.0)


def ref_embed_grad(ids, grad_out, rows, first, scale):
    """(sum, sum of absolute values, tokens) per row, in float64."""
    row = ids.cpu().long() - first
    here = (row >= 0) & (row < rows)
    row, x = row[here], grad_out.cpu().double()[here] * scale
    total = torch.zeros(rows, grad_out.shape[1], dtype=torch.float64)
    size = torch.zeros_like(total)
    total.index_add_(0, row, x)
    size.index_add_(0, row, x.abs())
    return total, size, torch.bincount(row, minlength=rows)


def embed_grad_bound(total, size, count, old, dtype):
    """n terms summed in any order are off by at most (n - 1) u times the sum
    of their sizes (to first order; 1 % on top covers the second); the scale's
    rounding, its product and the addition of `old` are three roundings more,
    and the result is rounded to the output type."""
    result = total if old is None else total + old
    err = 1.01 * U * (count.double()[:, None] + 2) * size + 1.01 * U * result.abs()
    return err + half_step(dtype) * (result.abs() + err) + 1e-40


# ---- distillation ------------------------------------------------------------------

def ref_distill(s, ids, u, tau, alpha, scale, mass=None, labels=None, row_grad=None):
    """Losses, lse, counted rows and gradient in float64, and the bounds of
    what fp32 may be off: a dict."""
    s = s.cpu().double()
    T, V = s.shape
    loss = torch.zeros(T, dtype=torch.float64)
    lse = torch.zeros(T, 2, dtype=torch.float64)
    counts = torch.zeros(T, dtype=torch.bool)
    grad = torch.zeros(T, V, dtype=torch.float64)
    loss_err = torch.zeros_like(loss)
    lse_err = torch.zeros_like(lse)
    grad_err = torch.zeros_like(grad)
    for t in range(T):
        label = None
        if labels is not None:
            label = int(labels[t])
            if not 0 <= label < V:
                continue
        n, top = 0, 0.0
        if alpha > 0 and ids is not None:
            value = u[t].double()
            there = (ids[t] >= 0) & (ids[t] < V) & (value != -math.inf)
            at, value = ids[t][there].long(), value[there]
            n = at.numel()
        if alpha == 1.0 and n == 0:
            continue
        counts[t] = True
        x = s[t]
        z = x / tau
        lse[t, 0] = torch.logsumexp(z, 0)
        q = torch.exp(z - lse[t, 0])
        w = torch.zeros(V, dtype=torch.float64)
        kd, total, ksum = 0.0, 0.0, 0.0
        if n:
            uz = value / tau
            top = float(uz.abs().max())
            norm = torch.logsumexp(uz, 0) if mass is None else mass[t].double().cpu()
            logp = uz - norm
            p = torch.exp(logp)
            w.index_add_(0, at, p)
            term = torch.where(p > 0, logp - (z[at] - lse[t, 0]), 0.0)
            kd = float((p * term).sum())
            # sizes of the numbers the fp32 form subtracts
            size = term.abs() + logp.abs() + z[at].abs() + lse[t, 0].abs()
            ksum = float(torch.where(p > 0, p * size, 0.0).sum())
            total = float(p.sum())
        loss[t] = alpha * tau * tau * kd
        slope = alpha * tau * (total * q - w)
        q1 = torch.zeros_like(q)
        hit = torch.zeros_like(q)
        if alpha < 1.0:
            lse[t, 1] = torch.logsumexp(x, 0)
            q1 = torch.exp(x - lse[t, 1])
            hit[label] = 1.0
            loss[t] += (1 - alpha) * (lse[t, 1] - x[label])
            slope = slope + (1 - alpha) * (q1 - hit)
        g = scale * (1.0 if row_grad is None else float(row_grad[t]))
        grad[t] = g * slope

        # A sum of exponentials: each exponent carries its subtraction, two
        # products and the factor's rounding (4 u of its size, at most the
        # spread of the finite logits), the exponential 2 u, the sum at most
        # one rounding for each of a thread's terms plus 64 for the joins.
        fin = x[torch.isfinite(x)]
        spread = float(fin.max() - fin.min()) if fin.numel() else 0.0
        # terms more than 110 below the maximum in log are below 2^-149
        d0, d1 = min(spread / tau, 110.0), min(spread, 110.0)
        sum0, sum1 = (4 * d0 + 2 + V / 64 + 64) * U, (4 * d1 + 2 + V / 64 + 64) * U
        size0 = abs(float(lse[t, 0])) + abs(float(z[torch.isfinite(z)].max())) if fin.numel() else 0
        size1 = abs(float(lse[t, 1])) + abs(float(fin.max())) if fin.numel() else 0
        lse_err[t, 0] = sum0 + 6 * U * size0
        lse_err[t, 1] = (sum1 + 6 * U * size1) if alpha < 1.0 else 0.0
        # log p: the quotient by tau, the norm (a log of a sum of K), the
        # difference; p adds the exponential
        logp_err = (8 * top + n + 16) * U
        kd_err = total * (logp_err + float(lse_err[t, 0])) + (logp_err + (8 + n) * U) * ksum
        loss_err[t] = alpha * tau * tau * kd_err + 8 * U * abs(float(loss[t]))
        if alpha < 1.0:
            loss_err[t] += (1 - alpha) * (float(lse_err[t, 1])
                                          + 4 * U * (abs(float(x[label])) + size1))
        # gradient: each softmax value (the exponent's error grows with the
        # distance of the logit from lse, at most log V more than the spread),
        # the taken share
        rel0 = float(lse_err[t, 0]) + (4 * (d0 + math.log(V)) + 16) * U + logp_err
        rel1 = float(lse_err[t, 1]) + (4 * (d1 + math.log(V)) + 16) * U
        grad_err[t] = abs(g) * (alpha * tau * (total * q * rel0 + w * (logp_err + 8 * U))
                                + (1 - alpha) * (q1 * rel1 + hit * 4 * U))
        grad_err[t] += 4 * U * grad[t].abs()
        # values whose exponential is below the smallest normal number are 0
        grad_err[t] += abs(g) * (alpha * tau * max(total, 1.0) + 1) * 2.0 ** -120
    return dict(loss=loss, lse=lse, counts=counts, grad=grad, loss_err=loss_err, lse_err=lse_err,
                grad_err=grad_err)


def assert_close(name, got, want, err, dtype):
    """|got - want| <= err, plus the output's rounding; NaN where want is."""
    got = got.cpu().double()
    bound = err + half_step(dtype) * (want.abs() + err) + 1e-40
    nan = torch.isnan(want)
    assert bool((torch.isnan(got) == nan).all()), f"{name}: NaN in other places"
    same = got == want                                   # infinities
    off = torch.where(same | nan, 0.0, (got - want).abs())
    bound = torch.where(same | nan, 1.0, bound)
    worst = float((off / bound).max()) if off.numel() else 0.0
    assert worst <= 1.0, f"{name}: {worst:.3g} times the bound"
    return worst
