"""distill_grad from a given lse: exp(s / tau - lse) as the formula has it, also
where lse is so large that lse * tau is no fp32 number."""
import pytest
import torch

import fsdp_sharded_optimizer_zero_amd as Z
from vocab_util import KIND, U, assert_close

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
