"""Distillation loss and gradient on the GPU against plain 64-bit forms."""
import math

import pytest
import torch

import fsdp_sharded_optimizer_zero_amd as Z
from vocab_util import KIND, U, assert_close, assert_guards, guarded, half_step, ref_distill

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
I32, I64 = torch.int32, torch.int64


class Problem:
    def __init__(self, rows, vocab, k, dtype=BF16, teacher=F32, idt=I64, tau=1.0, alpha=1.0,
                 scale=1.0, labels=True, mass=False, row_grad=False, pad=0, seed=1):
        g = torch.Generator().manual_seed(seed)
        self.rows, self.vocab, self.k = rows, vocab, k
        self.dtype, self.tau, self.alpha, self.scale, self.pad = dtype, tau, alpha, scale, pad
        s = torch.randn((rows, vocab), generator=g) * 2
        ids = torch.randint(0, vocab, (rows, max(k, 1)), generator=g)[:, :k]   # may repeat
        u = torch.randn((rows, k), generator=g) * 2 + 6
        if k:
            s.scatter_(1, ids, u + torch.randn((rows, k), generator=g))
            drop = torch.rand((rows, k), generator=g)
            ids = torch.where(drop < 0.1, -1, ids)
            ids = torch.where(drop > 0.95, vocab + 3, ids)
        self.buf, self.s = guarded(rows, vocab, vocab + pad, dtype, float("nan"))
        self.s.copy_(s)
        self.ids = ids.to(idt).cuda()
        self.u = u.to(teacher).cuda()
        self.mass = (torch.logsumexp(u.to(teacher).float() / tau, 1) + 0.1).cuda() \
            if mass and k else None
        self.labels = None
        if labels:
            lab = torch.randint(0, vocab, (rows,), generator=g)
            if rows > 2:
                lab[torch.rand(rows, generator=g) < 0.2] = -100
                lab[rows // 2] = vocab
            self.labels = lab.to(idt).cuda()
        self.row_grad = (torch.randn(rows, generator=g)).cuda() if row_grad else None
        self.desc = Z.make_distill(rows, vocab, k, logits_pitch=vocab + pad,
                                   grad_pitch=vocab + 2 * pad, logits_dtype=KIND[dtype],
                                   teacher_dtype=KIND[teacher], id_dtype=KIND[idt],
                                   temperature=tau, alpha=alpha, scale=scale)

    def ref(self):
        rg = None if self.row_grad is None else self.row_grad.cpu()
        return ref_distill(self.s, self.ids.cpu(), self.u.cpu(), self.tau, self.alpha, self.scale,
                           self.mass, None if self.labels is None else self.labels.cpu(), rg)

    def run(self, calls, in_place=False, sums=True):
        d, n = self.desc, self.rows
        need = Z.zs_distill_workspace_bytes(d)
        ws = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device="cuda")
        loss = torch.full((n + 1,), -7.0, device="cuda")
        lse = torch.full((2 * n + 1,), -7.0, device="cuda")
        total = torch.full((1,), -7.0, device="cuda") if sums else None
        count = torch.full((1,), -7, dtype=I64, device="cuda") if sums else None
        gbuf, grad = guarded(n, self.vocab, self.vocab + 2 * self.pad, self.dtype)
        if in_place:
            d = Z.zs_distill.from_buffer_copy(d)
            d.grad_pitch = d.logits_pitch
            store = self.s.clone()
            gbuf, grad = self.buf, self.s
        kw = dict(teacher_lse=self.mass, labels=self.labels)
        more = dict(loss_sum=total, counted=count, workspace=ws, workspace_bytes=need)
        if calls == "step":
            Z.distill_loss_grad(d, self.s, self.ids, self.u, loss[:n], grad, lse=lse[:2 * n],
                                row_grad=self.row_grad, **kw, **more)
        else:
            Z.distill_loss(d, self.s, self.ids, self.u, loss[:n], lse[:2 * n], **kw, **more)
            if calls == "pair":
                Z.distill_grad(d, self.s, self.ids, self.u, lse[:2 * n], grad,
                               row_grad=self.row_grad, **kw)
        torch.cuda.synchronize()
        assert bool((ws[need:] == 0x5A).all()), "written behind the workspace"
        assert float(loss[n]) == -7.0 and float(lse[2 * n]) == -7.0
        out = dict(loss=loss[:n], lse=lse[:2 * n].view(n, 2), total=total, count=count)
        if calls != "loss":
            out["grad"] = grad.clone()
            if in_place:
                self.s.copy_(store)
            else:
                assert_guards(gbuf, n, self.vocab, self.vocab + 2 * self.pad)
        return out

    def check(self, calls, ref=None, **kw):
        r = self.ref() if ref is None else ref
        o = self.run(calls, **kw)
        assert_close("loss", o["loss"], r["loss"], r["loss_err"], F32)
        assert_close("lse", o["lse"], r["lse"], r["lse_err"], F32)
        if o["total"] is not None:
            assert int(o["count"]) == int(r["counts"].sum())
            assert_close("loss_sum", o["total"], r["loss"].sum().reshape(1),
                         r["loss_err"].sum().reshape(1) + r["loss"].abs().sum() * U, F32)
        if calls != "loss":
            # the pair's gradient starts from an lse rounded to fp32
            err = r["grad_err"]
            assert_close("grad", o["grad"], r["grad"], err, self.dtype)
            masked = o["grad"].cpu()[~r["counts"]]
            assert bool((masked == 0).all())
        return o


# long rows up to 127 of them are cut into parts, 128 and more (and short ones) take one block each
SIZES = [(1, 1, 1), (1, 7, 3), (2, 8, 8), (3, 9, 1), (5, 1000, 16), (2, 50257, 64), (1, 131075, 130),
         (40, 12345, 33), (513, 61, 5), (515, 4097, 20)]


@pytest.mark.parametrize("rows,vocab,k", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("alpha", [1.0, 0.6])
@pytest.mark.parametrize("calls", ["loss", "pair", "step"])
def test_sizes(rows, vocab, k, dtype, alpha, calls):
    Problem(rows, vocab, k, dtype, tau=2.0, alpha=alpha, scale=0.25).check(calls)


@pytest.mark.parametrize("rows", [6, 520])
@pytest.mark.parametrize("calls", ["pair", "step"])
@pytest.mark.parametrize("teacher,idt,tau,mass,row_grad,pad", [
    (BF16, I32, 1.0, False, True, 0), (F32, I32, 4.0, True, False, 5), (BF16, I64, 0.5, True, True, 8),
    (F32, I64, 1.5, False, False, 3)])
def test_forms(rows, calls, teacher, idt, tau, mass, row_grad, pad):
    for dtype in (BF16, F32):
        for alpha, labels in ((1.0, False), (1.0, True), (0.3, True)):
            Problem(rows, 777, 12, dtype, teacher, idt, tau, alpha, 0.5, labels, mass, row_grad,
                    pad).check(calls)


@pytest.mark.parametrize("rows", [4, 513])
@pytest.mark.parametrize("calls", ["pair", "step"])
def test_labels_alone(rows, calls):
    """alpha = 0: the cross entropy of the labels; no teacher is read."""
    p = Problem(rows, 1001, 0, F32, alpha=0.0, scale=2.0)
    p.check(calls)
    q = Problem(rows, 1001, 4, F32, alpha=0.0, scale=2.0)
    q.ids, q.u = None, None
    o = q.run(calls)
    r = ref_distill(q.s, None, None, 1.0, 0.0, 2.0, None, q.labels.cpu())
    assert_close("loss", o["loss"], r["loss"], r["loss_err"], F32)
    assert_close("grad", o["grad"], r["grad"], r["grad_err"], F32)


@pytest.mark.parametrize("rows", [3, 512])
@pytest.mark.parametrize("k", [1023, 1024])
def test_most_entries_and_repeats(rows, k):
    """Far more entries than columns: every column several times."""
    for vocab in (5, 300, 20011):
        Problem(rows, vocab, k, F32, tau=2.0, alpha=0.5).check("step")


@pytest.mark.parametrize("rows", [3, 600])
@pytest.mark.parametrize("k", [63, 64, 65, 127, 128, 129, 300])
def test_entries_past_one_wave(rows, k):
    """Columns once, twice and more often, and the same bits on every run."""
    for vocab, dtype in ((101, F32), (20011, BF16), (40009, F32)):
        p = Problem(rows, vocab, k, dtype, tau=2.0, alpha=0.5, pad=1)
        p.ids[:, k // 2] = p.ids[:, 0]                     # a pair of every row's
        p.ids[:, k // 3] = p.ids[:, 1]
        p.ids[:, k - 1] = p.ids[:, 1]                      # and three of a column
        keep = p.labels >= 0
        keep &= p.labels < vocab
        p.labels[keep] = p.ids[keep, 2].clamp(0, vocab - 1)  # the label's is an entry's too
        ref = p.ref()
        for calls in ("pair", "step"):
            a, b = p.check(calls, ref), p.run(calls)
            assert torch.equal(a["grad"], b["grad"]) and torch.equal(a["loss"], b["loss"])


@pytest.mark.parametrize("rows", [5, 600])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("calls", ["pair", "step"])
def test_in_place(rows, dtype, calls):
    p = Problem(rows, 3001, 9, dtype, alpha=0.5, tau=2.0, pad=3)
    ref = p.ref()
    a = p.check(calls, ref)
    b = p.check(calls, ref, in_place=True)
    assert torch.equal(a["grad"], b["grad"]) and torch.equal(a["loss"], b["loss"])


@pytest.mark.parametrize("rows", [8, 520])
@pytest.mark.parametrize("alpha", [1.0, 0.5])
@pytest.mark.parametrize("calls", ["pair", "step"])
def test_masked_places(rows, alpha, calls):
    """Rows that do not count may hold anything; masked columns (-Inf, or the
    type's lowest value) have probability 0; an entry of -Inf is none."""
    p = Problem(rows, 515, 10, F32, alpha=alpha, tau=2.0)
    p.labels[0], p.labels[1] = -100, p.vocab
    p.s[0] = math.nan
    p.s[1, ::2] = math.inf
    p.labels[2], p.labels[3], p.labels[4] = 7, 8, 9
    p.ids[3] = -1                                  # no entry: counts only with alpha < 1
    p.u[4] = -math.inf
    keep = torch.zeros(p.vocab, dtype=torch.bool, device="cuda")
    keep[7:10] = True
    for t in (2, 5):
        row = keep.clone()
        row[p.ids[t][(p.ids[t] >= 0) & (p.ids[t] < p.vocab)].long()] = True
        row[100:110] = True
        p.s[t, ~row] = -math.inf if t == 2 else torch.finfo(F32).min
    p.ids[2, 0], p.u[2, 0] = 200, -math.inf        # a masked column at an entry that is none
    p.check(calls)


@pytest.mark.parametrize("rows", [4, 520])
def test_nan_and_infinities_in_rows_that_count(rows):
    """They reach that row alone; a teacher that wants a masked column makes
    the loss infinite and leaves the gradient finite."""
    p = Problem(rows, 300, 4, F32, labels=False, tau=1.0)
    p.ids[:] = torch.tensor([1, 5, 9, 250]).cuda()
    p.s[0, 17] = math.nan
    p.s[1, 9] = -math.inf
    o = p.run("step")
    assert math.isnan(float(o["loss"][0])) and bool(torch.isnan(o["grad"][0]).all())
    assert float(o["loss"][1]) == math.inf
    assert float(o["grad"][1, 9]) < 0 and bool(torch.isfinite(o["grad"][1]).all())
    assert bool(torch.isfinite(o["grad"][2:]).all()) and bool(torch.isfinite(o["loss"][2:]).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_large_and_constant_logits(dtype):
    """No overflow far from zero, where exp alone would; equal logits."""
    p = Problem(6, 999, 3, dtype, labels=False)
    p.s[0], p.s[1], p.s[2] = 3e38, -3e38, 0.0
    p.s[3] += 1e4
    p.check("step")
    p.check("pair")


@pytest.mark.parametrize("dtype,vocab", [(BF16, 140003), (F32, 70001), (BF16, 131072), (F32, 40005)])
@pytest.mark.parametrize("alpha,tau", [(1.0, 1.0), (0.5, 2.0), (0.5, 1.0)])
def test_long_rows_one_block_each(dtype, vocab, alpha, tau):
    """Rows as long as a block holds, and longer; among them one with masked
    columns, one of equal lowest values, one far from zero."""
    rows = 512
    p = Problem(rows, vocab, 20, dtype, alpha=alpha, tau=tau, pad=1)
    use = [0, 3, 200, 201, 510, 511]
    p.labels[:] = -100
    for t in use:
        p.labels[t] = 11 * t % vocab
    low = torch.finfo(dtype).min
    p.s[3, 100:vocab - 7] = low
    p.ids[3] = torch.arange(20).cuda()
    p.labels[3] = 5
    p.s[200] = low
    p.s[201] = (p.s[201].float() + 3e5).to(dtype)
    p.s[510, ::3] = -math.inf
    p.ids[510] = 3 * torch.arange(20).cuda() + 1
    p.labels[510] = 31
    ref = p.ref()
    a = p.check("step", ref)
    p.check("pair", ref)
    b = p.run("step", in_place=True)
    assert torch.equal(a["grad"], b["grad"]) and torch.equal(a["loss"], b["loss"])


@pytest.mark.parametrize("rows", [6, 127, 128])
@pytest.mark.parametrize("dtype,vocab", [(BF16, 50003), (F32, 40005), (BF16, 8199), (F32, 4103)])
@pytest.mark.parametrize("alpha,tau", [(1.0, 1.0), (0.5, 2.0), (0.5, 1.0)])
def test_masked_places_in_parts(rows, dtype, vocab, alpha, tau):
    """Whole parts masked by -Inf or the type's lowest value, masked rows, a
    row without entries, at row counts around the two ways to cut the work."""
    p = Problem(rows, vocab, 12, dtype, alpha=alpha, tau=tau, pad=1)
    p.labels[:] = torch.arange(rows).cuda() * 13 % vocab
    p.labels[0], p.s[0] = -100, math.nan
    low = torch.finfo(dtype).min
    for t, masked in ((1, -math.inf), (2, low)):
        p.s[t, 40:vocab - 3] = masked                  # what is left is at both ends
        p.ids[t] = torch.arange(12).cuda()
        p.labels[t] = vocab - 1
    p.ids[3] = -1
    p.s[4, :-2] = -math.inf                            # the last part alone has any
    p.ids[4] = vocab - 1
    p.labels[4] = vocab - 2
    ref = p.ref()
    for calls in ("pair", "step"):
        a, b = p.check(calls, ref), p.run(calls, in_place=True)
        assert torch.equal(a["grad"], b["grad"]) and torch.equal(a["loss"], b["loss"])


@pytest.mark.parametrize("rows", [3, 513])
@pytest.mark.parametrize("tau", [0.5, 2.0])
def test_teacher_entries_all_at_the_lowest_value(rows, tau):
    """Equal entries are equally likely, at the type's lowest value too."""
    p = Problem(rows, 200, 5, F32, labels=False, tau=tau)
    p.u[0] = torch.finfo(F32).min
    p.u[1] = torch.finfo(F32).max
    p.ids[:2] = torch.tensor([3, 50, 60, 70, 199]).cuda()
    o = p.run("step")
    q = p.u.clone()
    q[:2] = 0.0                          # the same distribution
    p.u = q
    p.check("step")
    want = p.run("step")
    # log p: the same five numbers, up to rounding of equal operations
    assert torch.equal(o["loss"], want["loss"]) and torch.equal(o["grad"], want["grad"])


def test_accumulate_and_no_rows():
    p = Problem(9, 100, 4, F32)
    r = p.ref()
    ws = torch.empty(Z.zs_distill_workspace_bytes(p.desc), dtype=torch.uint8, device="cuda")
    loss, lse = torch.empty(9, device="cuda"), torch.empty((9, 2), device="cuda")
    total = torch.full((1,), 2.5, device="cuda")
    count = torch.full((1,), 40, dtype=I64, device="cuda")
    Z.distill_loss(p.desc, p.s, p.ids, p.u, loss, lse, labels=p.labels, loss_sum=total,
                   counted=count, accumulate=True, workspace=ws)
    assert int(count) == 40 + int(r["counts"].sum())
    want = 2.5 + float(r["loss"].sum())
    assert abs(float(total) - want) <= float(r["loss_err"].sum()) + 16 * U * abs(want)
    # no rows: the sums are still set, or left
    d = Z.make_distill(0, 100, 4, logits_dtype=Z.ZS_F32)
    ws = torch.empty(Z.zs_distill_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    Z.distill_loss(d, None, None, None, None, None, loss_sum=total, counted=count, accumulate=True,
                   workspace=ws)
    assert int(count) == 40 + int(r["counts"].sum()) and abs(float(total) - want) < 1
    Z.distill_loss_grad(d, None, None, None, None, None, loss_sum=total, counted=count,
                        workspace=ws)
    assert int(count) == 0 and float(total) == 0.0


@pytest.mark.parametrize("rows", [7, 530])
def test_same_bits_and_both_orders_agree(rows):
    """Run to run the same bits; the one-call gradient and the pair's differ
    by no more than the bounds of both."""
    p = Problem(rows, 4099, 17, F32, alpha=0.4, tau=3.0, mass=True)
    a, b = p.run("step"), p.run("step")
    for name in ("loss", "lse", "grad", "total", "count"):
        assert torch.equal(a[name], b[name])
    c = p.run("pair")
    assert torch.equal(a["loss"], c["loss"]) and torch.equal(a["lse"], c["lse"])
    err = p.ref()["grad_err"]
    off = (a["grad"].cpu().double() - c["grad"].cpu().double()).abs()
    assert bool((off <= 2 * (err + half_step(F32) * a["grad"].cpu().abs()) + 1e-40).all())


def test_gradient_matches_differences():
    """Central differences of the 64-bit loss at the GPU's gradient."""
    p = Problem(2, 50, 6, F32, tau=2.0, alpha=0.5, labels=False)
    p.labels = torch.tensor([3, 44]).cuda()
    o = p.run("step")

    def f(s):
        return float(ref_distill(s, p.ids.cpu(), p.u.cpu(), 2.0, 0.5, 1.0, None,
                                 p.labels.cpu())["loss"].sum())

    s = p.s.cpu().double()
    h = 1e-4
    for t, v in [(0, 3), (0, 10), (1, 44), (1, int(p.ids[1].clamp(0, 49)[2]))]:
        up, down = s.clone(), s.clone()
        up[t, v] += h
        down[t, v] -= h
        d = (f(up) - f(down)) / (2 * h)
        # third derivatives are below 4 here: h^2 / 6 * 4, and fp32 gradients
        assert abs(d - float(o["grad"][t, v])) <= 1e-8 + 1e-5 * max(1.0, abs(d))


def test_logits_offsets_past_32_bits():
    """Rows whose element offsets pass 2^32."""
    vocab, pitch = 300, (1 << 31) + 40
    p = Problem(3, vocab, 4, BF16, labels=False)
    big = torch.empty(2 * pitch + vocab, dtype=BF16, device="cuda")
    view = big.as_strided((3, vocab), (pitch, 1))
    view.copy_(p.s)
    want = p.run("step")
    d = Z.make_distill(3, vocab, 4, logits_pitch=pitch, grad_pitch=pitch)
    ws = torch.empty(Z.zs_distill_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    loss = torch.empty(3, device="cuda")
    Z.distill_loss_grad(d, big, p.ids, p.u, loss, big, workspace=ws)
    assert torch.equal(loss, want["loss"]) and torch.equal(view, want["grad"])


@pytest.mark.parametrize("rows", [70, 900])
def test_smallgrid_build_matches(rows):
    p = Problem(rows, 20000, 8, BF16, alpha=0.5)
    a = p.run("step")
    with Z.library(Z.SMALLGRID_LIB_PATH):
        b = p.run("step")
        c = p.run("pair")
    for name in ("loss", "lse", "grad", "total", "count"):
        assert torch.equal(a[name], b[name]), name
    assert torch.equal(a["loss"], c["loss"])


def test_binding_refusals():
    p = Problem(4, 64, 2, BF16)
    ws = torch.empty(Z.zs_distill_workspace_bytes(p.desc), dtype=torch.uint8, device="cuda")
    good = dict(logits=p.s, ids=p.ids, u=p.u, loss=torch.empty(4, device="cuda"),
                lse=torch.empty((4, 2), device="cuda"), labels=p.labels)
    for bad in (dict(logits=p.s.float()), dict(logits=p.s[:3]), dict(ids=p.ids.int()),
                dict(u=p.u[:, :1].contiguous()), dict(u=p.u.half()), dict(loss=good["loss"][:3]),
                dict(lse=good["loss"]), dict(labels=p.labels.cpu()), dict(labels=p.labels[:2])):
        kw = good | bad
        with pytest.raises(ValueError):
            Z.distill_loss(p.desc, kw["logits"], kw["ids"], kw["u"], kw["loss"], kw["lse"],
                           labels=kw["labels"], workspace=ws)
    with pytest.raises(Z.ZSError) as err:
        Z.distill_loss(p.desc, p.s, p.ids, p.u, good["loss"], good["lse"], labels=p.labels,
                       workspace=ws[:-16])
    assert err.value.code == Z.ZS_EWORKSPACE
