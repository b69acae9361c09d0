"""The operators of many tensors and of the position table together, as a
training step uses them: a model whose small parameters are kept whole beside
the sharded vocabulary table."""
import math

import pytest
import torch

import fsdp_sharded_optimizer_zero_amd as Z
from fsdp_sharded_optimizer_zero_amd.runner import RelposBias, TableBatch, TableRun
from relpos_util import U, ref_bias, ref_grad

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


class Mixer:
    """Attention by position alone: every head mixes its part of the hidden
    states over the earlier tokens of a sequence, with weights from the bias
    table; then a learned scale.  Keeps what the calls saw."""

    def __init__(self, sequences, length, heads):
        self.shape, self.heads = (sequences, length), heads
        self.r = Z.make_relpos(heads, length, length, batch=sequences, bidirectional=False,
                               causal=True, scale=0.5, table_dtype=Z.ZS_BF16, dtype=Z.ZS_F32,
                               buckets=8, max_distance=20)
        self.lengths = None

    def __call__(self, hidden, bias, gain):
        s, n = self.shape
        x = hidden.float().view(s, n, self.heads, -1).transpose(1, 2).contiguous()
        scores = torch.matmul(x, x.transpose(2, 3).contiguous())
        biased = RelposBias.apply(self.r, bias, scores, self.lengths)
        self.seen = (bias, scores, biased)
        if biased.requires_grad:
            biased.register_hook(lambda g: setattr(self, "grad", g.clone()))
        mixed = torch.matmul(torch.softmax(biased, dim=3), x)
        mixed = mixed.transpose(1, 2).reshape(s * n, -1)
        return (hidden.float() + mixed * gain.float()).to(BF16)


def make_batch(tokens, rows, k, seed):
    g = torch.Generator().manual_seed(seed)
    labels = torch.randint(0, rows, (tokens,), generator=g)
    labels[torch.rand(tokens, generator=g) < 0.2] = -100
    return TableBatch(ids=torch.randint(0, rows, (tokens,), generator=g).cuda(),
                      teacher_ids=torch.randint(0, rows, (tokens, k), generator=g).cuda(),
                      teacher_logits=(torch.randn((tokens, k), generator=g) * 2).cuda(),
                      labels=labels.cuda(), valid=int((labels >= 0).sum()))


@pytest.mark.parametrize("max_norm", [1e-3, 100.0])
def test_step(max_norm):
    n_d, rows, dim, k, heads = 3, 90, 24, 5, 4
    seqs, length = 4, 17
    tokens = seqs * length
    mix = Mixer(seqs, length, heads)
    g = torch.Generator().manual_seed(1)
    whole = [torch.randn((8, heads), generator=g) * 0.3, torch.ones(dim)]
    run = TableRun(rows, dim, n_d, tokens, k, alpha=0.6, body=mix, whole=whole,
                   max_grad_norm=max_norm)
    run.load((torch.randn((rows, dim), generator=g) * 0.3).cuda())
    assert torch.equal(run.whole[0].cpu(), whole[0].to(BF16))
    for t in (1, 2):
        batches = [make_batch(tokens, rows, k, 10 * t + r) for r in range(n_d)]
        for r, b in enumerate(batches):
            run.rank_pass(r, b)
            bias, scores, biased = mix.seen
            want, size = ref_bias(mix.r, bias.detach(), scores.detach(), None, None)
            got = biased.detach().cpu().double()
            fine = torch.isfinite(want)
            assert torch.equal(fine, torch.isfinite(got))
            assert bool(((got - want)[fine].abs() <= 2 * U * size[fine]).all())
            total, size, _ = ref_grad(mix.r, mix.grad, None, None)
            off = (run.rank_grads[r][0].cpu().double() - total).abs()
            assert bool((off <= 64 * U * size + 2.0 ** -8 * (total.abs() + 64 * U * size)).all())
        valid = [b.valid for b in batches]
        state = [x.clone() for x in run.whole_state]
        run.update(t, valid)
        # the mean over ranks, three products and sums in fp32
        for j, got in enumerate(run.whole_grads):
            parts = [run.rank_grads[r][j].cpu().double() * (valid[r] / sum(valid))
                     for r in range(n_d)]
            assert bool(((got.cpu().double() - sum(parts)).abs()
                         <= 8 * U * sum(p.abs() for p in parts) + 1e-40).all())
        # one norm over the shards and the whole tensors
        means = [m[:s.valid_len] for m, s in zip(run.mean, run.shards)]
        q = math.fsum((x.cpu().double() ** 2).sum().item() for x in means + run.whole_grads)
        assert abs(float(run.sqnorm) - q) <= 1e-12 * q
        c = min(1.0, max_norm / (math.sqrt(float(run.sqnorm)) + 1e-6))
        assert (c < 1.0) == (max_norm < 1.0)
        coef = torch.tensor(c, dtype=F32)
        n = run.whole_shard.valid_len
        flat = torch.cat([x.reshape(-1) for x in run.whole_grads])
        assert torch.equal(run.whole_mean[:n], flat * coef.cuda())
        # AdamW of the clipped gradient: some ten fp32 roundings of each value
        w, m, v = (x[:n].cpu().double() for x in state)
        gr = run.whole_mean[:n].cpu().double()
        m = 0.9 * m + 0.1 * gr
        v = 0.999 * v + 0.001 * gr * gr
        step = m / (1 - 0.9 ** t) / ((v / (1 - 0.999 ** t)).sqrt() + 1e-8) + 0.01 * w
        want = w - 1e-3 * step
        new = run.whole_state[0][:n].cpu().double()
        assert bool(((new - want).abs() <= 1e-6 * want.abs() + 1e-3 * 1e-4 * step.abs()
                     + 1e-12).all())
        assert torch.equal(run.whole_gather[:n], run.whole_state[0][:n].to(BF16))
        assert not torch.equal(new, w)


def test_relpos_function_gradients():
    """RelposBias against autograd of the plain form, in float64."""
    mix = Mixer(2, 13, 3)
    mix.r.table_dtype = Z.ZS_F32
    g = torch.Generator(device="cuda").manual_seed(2)
    scores = torch.randn((2, 3, 13, 13), generator=g, device="cuda", requires_grad=True)
    table = torch.randn((8, 3), generator=g, device="cuda", requires_grad=True)
    weight = torch.randn((2, 3, 13, 13), generator=g, device="cuda")
    lengths = torch.tensor([13, 6], device="cuda")
    out = RelposBias.apply(mix.r, table, scores, lengths)
    p = torch.softmax(out, dim=3)
    ds, dt = torch.autograd.grad((p * weight).sum(), [scores, table])
    from relpos_util import buckets_of, positions
    s64, t64 = scores.detach().cpu().double().requires_grad_(), \
        table.detach().cpu().double().requires_grad_()
    rows = []
    for b in range(2):
        d, seen = positions(mix.r, b, lengths, None)
        value = s64[b] * 0.5 + t64[buckets_of(mix.r, d)].permute(2, 0, 1)
        rows.append(value.masked_fill(~seen, -math.inf))
    p64 = torch.softmax(torch.stack(rows), dim=3)
    es, et = torch.autograd.grad((p64 * weight.cpu().double()).sum(), [s64, t64])
    # softmax's own fp32 error, a few u of values of size up to 4, summed over
    # at most 26 x 13 places
    assert float((ds.cpu().double() - es).abs().max()) < 64 * U * 4
    assert float((dt.cpu().double() - et).abs().max()) < 26 * 13 * 64 * U
    # the bias alone, and no gradient of scores
    alone = RelposBias.apply(mix.r, table)
    assert alone.shape == (2, 3, 13, 13)
    once = torch.autograd.grad(alone[torch.isfinite(alone)].sum(), table)[0]
    assert torch.equal(once.sum(0), torch.full((3,), 2.0 * 91, device="cuda"))


@pytest.mark.parametrize("none", [0.0, -1.0])
def test_step_without_a_clip(none):
    """max_grad_norm <= 0 is no clip: the same bits as a limit that is not reached."""
    n_d, rows, dim, k, heads = 2, 90, 24, 5, 4
    seqs, length = 4, 17
    runs = []
    for max_norm in (none, 1e6):
        g = torch.Generator().manual_seed(1)
        whole = [torch.randn((8, heads), generator=g) * 0.3, torch.ones(dim)]
        run = TableRun(rows, dim, n_d, seqs * length, k, alpha=0.6, body=Mixer(seqs, length, heads),
                       whole=whole, max_grad_norm=max_norm)
        run.load((torch.randn((rows, dim), generator=g) * 0.3).cuda())
        for t in (1, 2):
            run.step(t, [make_batch(seqs * length, rows, k, 10 * t + r) for r in range(n_d)])
            flat = torch.cat([x.reshape(-1) for x in run.whole_grads])
            assert torch.equal(run.whole_mean[:len(flat)], flat) and bool((flat != 0).any())
        runs.append(run)
    a, b = runs
    assert torch.equal(a.sqnorm, b.sqnorm) and torch.equal(a.gather, b.gather)
    assert torch.equal(a.whole_gather, b.whole_gather)
    for x, y in zip([a.whole_state, *a.state], [b.whole_state, *b.state]):
        assert all(torch.equal(u, v) for u, v in zip(x, y))


@pytest.mark.parametrize("shape,pitch", [((32, 6), 6), ((13, 5), 5), ((75,), 5)])
def test_relpos_function_gradient_of_unused_entries(shape, pitch):
    """A table with more rows or columns than the call uses: 0 for those."""
    r = Z.make_relpos(5, 9, 70, buckets=8, max_distance=20, dtype=Z.ZS_F32, table_pitch=pitch)
    table = torch.randn(shape, device="cuda", requires_grad=True)
    out = RelposBias.apply(r, table)
    # what the next allocations find
    stale = [torch.full(shape, math.nan, device="cuda") for _ in range(4)]
    del stale
    got = torch.autograd.grad(out.sum(), table)[0]
    assert got.shape == table.shape
    rows = got.view(-1, pitch)
    used = torch.zeros_like(rows, dtype=torch.bool)
    used[:8, :5] = True
    assert bool((rows[~used] == 0).all())
    assert torch.equal(rows[:8, :5].sum(0), torch.full((5,), 9.0 * 70, device="cuda"))


@pytest.mark.parametrize("extra", [0, 11])
def test_relpos_function_of_flat_scores(extra):
    """Scores as a flat buffer, and without the batch of one: the gradient has
    their shape, 0 behind the places."""
    r = Z.make_relpos(3, 9, 70, dtype=Z.ZS_F32, scale=0.5)
    n = 3 * 9 * 70
    table = torch.randn((32, 3), device="cuda", requires_grad=True)
    flat = torch.randn(n + extra, device="cuda", requires_grad=True)
    weight = torch.randn((1, 3, 9, 70), device="cuda")
    out = RelposBias.apply(r, table, flat)
    stale = [torch.full((n + extra,), math.nan, device="cuda") for _ in range(4)]
    del stale
    got = torch.autograd.grad((out * weight).sum(), flat)[0]
    assert got.shape == flat.shape and bool((got[n:] == 0).all())
    assert torch.equal(got[:n], (weight * 0.5).reshape(-1))
    three = flat.detach()[:n].view(3, 9, 70).requires_grad_()
    out3 = RelposBias.apply(r, table, three)
    assert torch.equal(out3, out)
    got = torch.autograd.grad((out3 * weight).sum(), three)[0]
    assert torch.equal(got, weight[0] * 0.5)


def test_relpos_function_when_the_table_changes():
    """The gradient does not depend on the table: it may be written between the
    passes, as an embedding's may.  The lengths are needed and may not."""
    r = Z.make_relpos(3, 9, 70, batch=2, dtype=Z.ZS_F32)
    table = torch.randn((32, 3), device="cuda", requires_grad=True)
    lengths = torch.tensor([70, 20], device="cuda")
    want = torch.autograd.grad(RelposBias.apply(r, table, None, lengths)[0].sum(), table)[0]
    out = RelposBias.apply(r, table, None, lengths)
    with torch.no_grad():
        table.mul_(2.0)
    assert torch.equal(torch.autograd.grad(out[0].sum(), table)[0], want)
    out = RelposBias.apply(r, table, None, lengths)
    lengths.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(out[0].sum(), table)
