"""Distillation of rows far from zero, held to the bounds of the same rows near
zero: the loss, and the gradient of the one-call form, depend on differences of
logits alone, and an offset that fp32 (or bf16) adds exactly changes no
difference.  So a wave or a part of a row that is lost, or counted twice, shows
where the general bounds, which grow with lse, would hide it."""
import math

import pytest
import torch

import fsdp_sharded_optimizer_zero_amd as Z
from vocab_util import KIND, U, assert_close, ref_distill

BF16, F32 = torch.bfloat16, torch.float32
# |m log2(e) / tau| up to which the kernels subtract in the fma; beyond it a
# row is read again and the difference taken first
LIMIT = 65536.0 * math.log(2.0)


def base_row(kind, vocab, dtype, g):
    """(logits near zero, the offset) of one row, both exact in `dtype` at
    every temperature a power of two."""
    if dtype == BF16:
        # 8 bits of mantissa: the next smaller logits have weight 0
        return -1024.0 * (torch.rand(vocab, generator=g) < 0.5).double(), 196608.0 * kind
    x = torch.randint(-64, 64, (vocab,), generator=g).double() / 8
    if kind == 0:
        # waves on both sides of the limit, at the same weights: 64 lanes'
        # vectors of 4 up to 45426.0, and up to 45427 + 2
        wave = torch.arange(vocab) // 256 % 2
        return x.abs() / 4 * (2 * wave - 1), 45426.0
    return x, 2.0 ** 20 * kind if abs(kind) == 1 else 131072.0


class Far:
    def __init__(self, rows, vocab, dtype, tau, alpha, pad=0, k=9, counted=8, kinds=(1, -1, 2, 0)):
        g = torch.Generator().manual_seed(vocab + rows)
        self.rows, self.vocab, self.dtype, self.tau, self.alpha = rows, vocab, dtype, tau, alpha
        use = sorted({int(i) for i in torch.linspace(0, rows - 1, counted)})
        self.base = torch.zeros((rows, vocab), dtype=torch.float64)
        self.labels = torch.full((rows,), -100)
        self.ids = torch.randint(0, vocab, (rows, k), generator=g)
        self.u = torch.randn((rows, k), generator=g)
        self.offset = torch.zeros(rows, dtype=torch.float64)
        for i, t in enumerate(use):
            kind = kinds[i % len(kinds)]
            if dtype == BF16 and kind not in (1, -1):
                kind = 1
            self.base[t], self.offset[t] = base_row(kind, vocab, dtype, g)
            # the entries and the label among the larger logits
            top = torch.nonzero(self.base[t] >= 0)[:, 0]
            self.ids[t] = top[torch.randint(0, top.numel(), (k,), generator=g)]
            self.labels[t] = top[int(torch.randint(0, top.numel(), (1,), generator=g))]
        self.s = self.base + self.offset[:, None]
        assert bool((self.s.to(dtype).double() == self.s).all())
        self.pad = pad
        self.desc = Z.make_distill(rows, vocab, k, logits_pitch=vocab + pad,
                                   grad_pitch=vocab + pad, logits_dtype=KIND[dtype],
                                   temperature=tau, alpha=alpha)

    def ref(self, base=None):
        return ref_distill(self.base if base is None else base, self.ids, self.u, self.tau,
                           self.alpha, 1.0, None, self.labels)


CASES = [(F32, 2.0, 0.5), (F32, 1.0, 0.5), (F32, 1.0, 1.0), (F32, 0.5, 1.0), (BF16, 1.0, 0.5),
         (BF16, 2.0, 1.0)]


@pytest.mark.parametrize("dtype,tau,alpha", CASES)
def test_bounds_are_narrow(dtype, tau, alpha):
    """A 32nd of a row's columns left out of its sums, or counted twice, is
    past the bounds of the loss and of the gradient's largest values."""
    p = Far(4, 70001, dtype, tau, alpha)
    r = p.ref()
    q = r["grad"]
    for w in (0.0, 2.0):
        z = p.base / tau
        weight = torch.ones_like(z)
        weight[:, 64:64 + p.vocab // 32] = w
        lse = torch.log((torch.exp(z) * weight).sum(1))
        off = alpha * tau * tau * (lse - r["lse"][:, 0]).abs()      # of the loss
        assert bool((off > 4 * r["loss_err"]).all())
        softmax = torch.exp(z - r["lse"][:, :1])
        at = softmax.argmax(1, keepdim=True)
        top = softmax.gather(1, at)[:, 0]
        moved = alpha * tau * top * torch.expm1((r["lse"][:, 0] - lse).abs())
        plain = ~torch.zeros_like(q, dtype=torch.bool).scatter_(1, p.ids, True).gather(1, at)[:, 0]
        assert bool(((moved > 4 * r["grad_err"].gather(1, at)[:, 0]) | ~plain).all())


def from_lse(p, lse):
    """The gradient as distill_grad defines it from a given lse, and its bound."""
    grad, err = torch.zeros_like(p.s), torch.zeros_like(p.s)
    for t in torch.nonzero(p.labels >= 0)[:, 0].tolist():
        u = p.u[t].double() / p.tau
        prob = torch.softmax(u, 0)
        w = torch.zeros(p.vocab, dtype=torch.float64).index_add_(0, p.ids[t], prob)
        z0, z1 = p.s[t] / p.tau - lse[t, 0], p.s[t] - lse[t, 1]
        q0 = torch.exp(z0)
        q1 = torch.exp(z1) if p.alpha < 1.0 else torch.zeros_like(z0)
        hit = torch.zeros_like(w)
        hit[p.labels[t]] = 1.0 if p.alpha < 1.0 else 0.0
        a, b = p.alpha * p.tau, 1.0 - p.alpha
        grad[t] = a * (q0 - w) + b * (q1 - hit)
        # each value of a softmax: three roundings of its exponent (exact
        # differences; 1 / tau is a power of two), 16 u of exponentials and
        # factors; the teacher's as in the general bound
        p_err = (8 * float(u.abs().max()) + u.numel() + 16) * U
        err[t] = a * (q0 * ((4 * z0.abs() + 16) * U + p_err) + w * (p_err + 8 * U)) \
            + b * (q1 * (4 * z1.abs() + 16) * U + hit * 4 * U) + 4 * U * grad[t].abs() + 2.0 ** -120
    return grad, err


# one block a row (64, 128, 256, 512 and 1024 threads, a row longer than a block
# holds) and rows in parts (of 2 vectors a thread and of 8)
SHAPES = [(9, 509), (130, 2003), (130, 4001), (130, 12345), (130, 30011), (130, 70001),
          (9, 50003), (127, 70002), (300, 70001)]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,vocab", SHAPES)
@pytest.mark.parametrize("dtype,tau,alpha", CASES)
def test_far_from_zero(rows, vocab, dtype, tau, alpha):
    p = Far(rows, vocab, dtype, tau, alpha, pad=3)
    r = p.ref()
    n = rows
    logits = torch.full((n, vocab + 3), math.nan, dtype=dtype)
    logits[:, :vocab] = p.s.to(dtype)
    logits = logits.cuda()
    ids, u, labels = p.ids.cuda(), p.u.cuda(), p.labels.cuda()
    ws = torch.empty(Z.zs_distill_workspace_bytes(p.desc), dtype=torch.uint8, device="cuda")
    near = torch.where(r["counts"][:, None], r["lse"], 0.0)
    shift = torch.where(r["counts"], p.offset, 0.0)
    want = near + torch.stack([shift / tau, shift if alpha < 1.0 else shift * 0], dim=1)
    for one_call in (True, False):
        loss, lse = torch.empty(n, device="cuda"), torch.empty((n, 2), device="cuda")
        out = torch.empty((n, vocab + 3), dtype=dtype, device="cuda")
        if one_call:
            Z.distill_loss_grad(p.desc, logits, ids, u, loss, out, lse=lse, labels=labels,
                                workspace=ws)
            grad, err = r["grad"], r["grad_err"]
        else:
            Z.distill_loss(p.desc, logits, ids, u, loss, lse, labels=labels, workspace=ws)
            Z.distill_grad(p.desc, logits, ids, u, lse, out, labels=labels)
            grad, err = from_lse(p, lse.cpu().double())
        assert_close("loss", loss, r["loss"], r["loss_err"], F32)
        # m / tau is exact: the sum with log(sum) is the one rounding of its size
        assert_close("lse", lse, want, r["lse_err"], F32)
        assert_close("grad", out[:, :vocab], grad, err, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [9, 130])
@pytest.mark.parametrize("vocab", [1003, 12345])
def test_small_temperature(rows, vocab):
    """Ordinary logits at tau = 2^-13: 8 + j / 8192 at that temperature are
    65536 + j, beyond the fma form."""
    tau = 2.0 ** -13
    p = Far(rows, vocab, F32, tau, 1.0, kinds=(1,))
    g = torch.Generator().manual_seed(vocab)
    p.base = torch.randint(0, 24, (rows, vocab), generator=g).double() * tau
    p.u = p.u * tau
    p.offset = torch.full((rows,), 8.0, dtype=torch.float64)
    p.s = p.base + 8.0
    assert 8.0 / tau > LIMIT
    r = p.ref()
    loss, lse = torch.empty(rows, device="cuda"), torch.empty((rows, 2), device="cuda")
    out = torch.empty((rows, vocab), device="cuda")
    ws = torch.empty(Z.zs_distill_workspace_bytes(p.desc), dtype=torch.uint8, device="cuda")
    logits, ids, u, labels = p.s.float().cuda(), p.ids.cuda(), p.u.cuda(), p.labels.cuda()
    Z.distill_loss_grad(p.desc, logits, ids, u, loss, out, lse=lse, labels=labels, workspace=ws)
    assert_close("loss", loss, r["loss"], r["loss_err"], F32)
    assert_close("grad", out, r["grad"], r["grad_err"], F32)
    Z.distill_loss(p.desc, logits, ids, u, loss, lse, labels=labels, workspace=ws)
    assert_close("loss", loss, r["loss"], r["loss_err"], F32)
    Z.distill_grad(p.desc, logits, ids, u, lse, out, labels=labels)
    grad, err = from_lse(p, lse.cpu().double())
    assert_close("grad", out, grad, err, F32)
