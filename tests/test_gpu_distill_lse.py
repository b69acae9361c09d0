"""distill_grad from a given lse: exp(s / tau - lse) as the formula has it, also
where lse is so large that lse * tau is no fp32 number."""
import pytest
import torch

import fsdp_sharded_optimizer_zero_amd as Z
from vocab_util import KIND, U, assert_close, half_step, ref_distill

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
INV = 0.75          # 1 / tau, exact in fp32, with a tau that is not


def rows_at(size, dtype, vocab):
    """(logits [n, vocab], lse [n]): every lse an fp32 number near that row's
    largest s / tau, at all distances that fp32 has there up to about 8."""
    at = torch.tensor(size, dtype=dtype).double()
    step = abs(float(at)) * (2.0 ** -7 if dtype == BF16 else 2.0 ** -23)
    g = torch.Generator().manual_seed(int(size) % 1000)
    s = at - step * torch.randint(0, 4, (vocab,), generator=g).double()
    s = s.to(dtype).double()
    s[0] = at
    z = INV * float(at)
    lse = torch.tensor([z + d for d in range(-8, 9)], dtype=torch.float64).float().unique()
    return s.repeat(lse.numel(), 1), lse


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("vocab", [61, 5003])
@pytest.mark.parametrize("size", [3.0e1, 2.0e4, 3.1e6, 5.3e7, -5.3e7, 1.7e8])
def test_from_a_given_lse(dtype, vocab, size):
    s, lse = rows_at(size, dtype, vocab)
    rows, tau = lse.numel(), 1.0 / INV
    d = Z.make_distill(rows, vocab, 1, logits_dtype=KIND[dtype], temperature=tau)
    ids = torch.full((rows, 1), 2).cuda()
    u = torch.zeros((rows, 1)).cuda()                   # one entry: p = 1
    both = torch.stack([lse, torch.zeros(rows)], dim=1).contiguous().cuda()
    grad = torch.empty((rows, vocab), dtype=dtype, device="cuda")
    Z.distill_grad(d, s.to(dtype).cuda(), ids, u, both, grad)
    z = INV * s - lse.double()[:, None]
    q = torch.exp(z)
    want = tau * q
    want[:, 2] -= tau
    # Relative error of tau q.  With m = lse tau rounded, (s - m) is exact or
    # its value is 0; its product with log2(e)/tau carries that constant's two
    # roundings and one of its own, and in the fma form one more: 4 u of
    # |s - m| / tau, which is |z| + |rest|, |rest| <= u |lse|.  Two hardware
    # exponentials and one of rest (2 u each), rest's own rounding (u |rest|)
    # and eight products: 16 u.
    rest = U * lse.double().abs()[:, None]
    err = tau * q * U * (16 + 4 * (z.abs() + rest) + rest)
    err[:, 2] += 8 * U * tau
    err += 2.0 ** -120
    assert_close("grad", grad, want, err, dtype)


@pytest.mark.parametrize("rows", [9, 130])
@pytest.mark.parametrize("vocab", [300, 10007])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tau,alpha", [(1.5, 1.0), (0.3, 0.5), (0.5, 1.0), (3.0, 0.5), (7.0, 1.0),
                                       (1.0, 0.5), (0.9, 0.0)])
def test_rows_at_the_ends_of_the_type(rows, vocab, dtype, tau, alpha):
    """Rows of one value far from zero, a mask that leaves nothing among them:
    in one call uniform; in two calls lse can hold no more than the value, and
    every probability is a number from 0 to 1."""
    ends = [torch.finfo(dtype).min, torch.finfo(dtype).max, -3e38, 2.5e38, -1e30, 7e12, -3e9, 5e8]
    s = torch.zeros((rows, vocab), dtype=dtype)
    value = torch.zeros(rows, dtype=torch.float64)
    for t in range(rows):
        s[t] = ends[t % len(ends)]
        value[t] = float(s[t, 0])
    ids = (torch.arange(4)[None, :] * 61 + torch.arange(rows)[:, None]) % vocab
    u = (torch.arange(4.0) / 2).repeat(rows, 1)
    labels = torch.arange(rows) * 17 % vocab
    ref = ref_distill(torch.zeros((rows, vocab)), ids, u, tau, alpha, 1.0, None, labels)
    d = Z.make_distill(rows, vocab, 4, logits_dtype=KIND[dtype], temperature=tau, alpha=alpha)
    ws = torch.empty(Z.zs_distill_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    loss, lse = torch.empty(rows, device="cuda"), torch.empty((rows, 2), device="cuda")
    grad = torch.empty((rows, vocab), dtype=dtype, device="cuda")
    x = (s.cuda(), ids.cuda(), u.cuda())
    Z.distill_loss_grad(d, *x, loss, grad, lse=lse, labels=labels.cuda(), workspace=ws)
    assert_close("loss", loss, ref["loss"], ref["loss_err"], F32)
    assert_close("grad", grad, ref["grad"], ref["grad_err"], dtype)
    one = lse.clone()
    Z.distill_loss(d, *x, loss, lse, labels=labels.cuda(), workspace=ws)
    Z.distill_grad(d, *x, lse, grad, labels=labels.cuda())
    assert_close("loss", loss, ref["loss"], ref["loss_err"], F32)
    # the value's quotient by tau (1 / tau rounded, and the product), at most
    # fp32's largest number; log(vocab) is below the rounding
    most = torch.finfo(F32).max
    for got in (one, lse):
        got = got.cpu().double()
        assert bool(torch.isfinite(got).all())
        off = (got[:, 0] - (value / tau).clamp(-most, most)).abs()
        assert bool((off <= 3 * U * (value / tau).abs() + 10).all())
        assert alpha == 1.0 or bool(((got[:, 1] - value).abs() <= U * value.abs() + 10).all())
    # each value of a softmax in [0, 1], what entries and label take off; 1e-5
    # for the fp32 operations, as everywhere, and the output's rounding
    got = grad.cpu().double()
    room = 1 + 1e-5 + 2 * half_step(dtype)
    take = torch.zeros((rows, vocab), dtype=torch.float64)
    if alpha > 0:
        take.scatter_add_(1, ids, alpha * tau * torch.softmax(u.double() / tau, 1))
    if alpha < 1:
        take.scatter_add_(1, labels[:, None], torch.full((rows, 1), 1 - alpha).double())
    slope = alpha * tau + (1 - alpha)
    assert bool(torch.isfinite(got).all())
    assert bool((got <= slope * room).all()) and bool((got >= -take * room).all())


@pytest.mark.parametrize("rows", [9, 130])
@pytest.mark.parametrize("vocab", [300, 10007])
@pytest.mark.parametrize("tau,alpha", [(1.0, 1.0), (1.0, 0.5), (1.5, 1.0), (0.5, 0.5), (3.0, 0.5)])
def test_no_number_stays_none(rows, vocab, tau, alpha):
    """A NaN or +Inf among a row's logits, and a row of -Inf alone, are NaN in
    both forms, in every column, and in no other row."""
    g = torch.Generator().manual_seed(vocab)
    s = torch.randn((rows, vocab), generator=g)
    s[0, vocab // 2] = float("nan")
    s[2, vocab - 1] = float("inf")
    s[4] = -float("inf")
    ids = torch.arange(4).repeat(rows, 1)
    labels = torch.full((rows,), 5)
    d = Z.make_distill(rows, vocab, 4, logits_dtype=Z.ZS_F32, temperature=tau, alpha=alpha)
    ws = torch.empty(Z.zs_distill_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    loss, lse = torch.empty(rows, device="cuda"), torch.empty((rows, 2), device="cuda")
    one, two = torch.empty((2, rows, vocab), device="cuda")
    x = (s.cuda(), ids.cuda(), torch.zeros((rows, 4)).cuda())
    Z.distill_loss_grad(d, *x, loss, one, labels=labels.cuda(), workspace=ws)
    Z.distill_loss(d, *x, loss, lse, labels=labels.cuda(), workspace=ws)
    Z.distill_grad(d, *x, lse, two, labels=labels.cuda())
    none = torch.zeros(rows, dtype=torch.bool)
    none[[0, 2, 4]] = True
    for grad in (one, two):
        nan = torch.isnan(grad).cpu()
        assert torch.equal(nan.all(1), none) and torch.equal(nan.any(1), none)
        assert bool(torch.isfinite(grad.cpu()[~none]).all())
