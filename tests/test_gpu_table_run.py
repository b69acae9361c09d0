"""The table operators together, as a training step uses them: each one's
output against its 64-bit form from the inputs it had, through the reduction
and the optimizer step to the table the next step reads; graph capture;
several streams and host threads."""
import math
import os
import subprocess
import sys
import threading

import pytest
import torch

import fsdp_sharded_optimizer_zero_amd as Z
from fsdp_sharded_optimizer_zero_amd.runner import TableBatch, TableRun
from vocab_util import (U, assert_close, embed_grad_bound, half_step, ref_distill, ref_embed_grad,
                        ref_lookup)

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def make_batch(tokens, rows, k, seed, masked=0.2):
    g = torch.Generator().manual_seed(seed)
    labels = torch.randint(0, rows, (tokens,), generator=g)
    labels[torch.rand(tokens, generator=g) < masked] = -100
    ids = torch.randint(0, rows, (tokens,), generator=g)
    ids[::7] = -1
    return TableBatch(ids=ids.cuda(),
                      teacher_ids=torch.randint(0, rows, (tokens, k), generator=g).cuda(),
                      teacher_logits=(torch.randn((tokens, k), generator=g) * 2).cuda(),
                      labels=labels.cuda(), valid=int((labels >= 0).sum()))


def body(h):
    return torch.tanh(h.float()).to(BF16) + h


@pytest.mark.parametrize("tokens,rows,dim,k", [(9, 31, 16, 4), (150, 300, 40, 8),
                                               (600, 1000, 24, 5)])
@pytest.mark.parametrize("f32_grads,alpha,fn", [(True, 0.7, None), (False, 1.0, body)])
def test_step(tokens, rows, dim, k, f32_grads, alpha, fn):
    n_d, scale = 3, math.sqrt(dim)
    run = TableRun(rows, dim, n_d, tokens, k, scale=scale, temperature=2.0, alpha=alpha,
                   f32_grads=f32_grads, body=fn)
    g = torch.Generator().manual_seed(3)
    run.load((torch.randn((rows, dim), generator=g) * 0.1).cuda())
    dtype = F32 if f32_grads else BF16
    scale32 = float(torch.tensor(scale, dtype=F32))
    for t in (1, 2):
        batches = [make_batch(tokens, rows, k, 10 * t + r, masked=1.0 if r == 1 else 0.2)
                   for r in range(n_d)]                  # rank 1 has only padding
        table = run.table.clone()
        loss = 0.0
        for r, b in enumerate(batches):
            run.rank_pass(r, b)
            want = ref_lookup(b.ids, table, 0, scale32)
            assert_close("hidden", run.hidden, want, want.abs() * U, BF16)
            ref = ref_distill(run.logits, b.teacher_ids.cpu(), b.teacher_logits.cpu(), 2.0, alpha,
                              1.0 / max(b.valid, 1), None, b.labels.cpu())
            assert_close("loss", run.loss[r], ref["loss"], ref["loss_err"], F32)
            assert_close("dlogits", run.dlogits, ref["grad"], ref["grad_err"], BF16)
            loss += float(ref["loss"].sum())
            # what embed_grad added to the head's gradient
            h = run.hidden if fn is None else fn(run.hidden)
            head = torch.mm(run.dlogits.t(), h).to(dtype).cpu().double()
            total, size, count = ref_embed_grad(b.ids, run.dhidden, rows, 0, scale32)
            off = (run.grad_table(r).cpu().double() - (total + head)).abs()
            assert bool((off <= embed_grad_bound(total, size, count, head, dtype)).all())
        valid = [b.valid for b in batches]
        assert int(run.counted) == sum(valid) and valid[1] == 0
        assert abs(float(run.loss_sum) - loss) <= 1e-4 * abs(loss)
        grads = run.grads[:, :rows * dim].double().cpu()
        w = [x[0].clone() for x in run.state]
        run.update(t, valid)
        mean = torch.zeros(rows * dim, dtype=torch.float64)
        for r in range(n_d):
            mean += grads[r] * (valid[r] / sum(valid))
        got = torch.cat([m[:s.valid_len] for m, s in zip(run.mean, run.shards)]).cpu().double()
        # three weights, products and sums in fp32
        sizes = sum(grads[r].abs() * (valid[r] / sum(valid)) for r in range(n_d))
        assert bool(((got - mean).abs() <= 6 * U * sizes + 1e-40).all())
        q = float((got ** 2).sum())
        assert abs(float(run.sqnorm) - q) <= 1e-12 * q
        # the gathered table is the bf16 rounding of the updated masters
        new = torch.cat([x[0][:s.valid_len] for x, s in zip(run.state, run.shards)])
        assert torch.equal(run.table.reshape(-1), new.to(BF16))
        assert any(not torch.equal(a, x[0]) for a, x in zip(w, run.state))


class Calls:
    """The four kinds of calls on one set of buffers."""

    def __init__(self, tokens, rows, dim, k, seed):
        g = torch.Generator().manual_seed(seed)
        self.b = make_batch(tokens, rows, k, seed)
        self.table = (torch.randn((rows, dim), generator=g) * 0.1).to(BF16).cuda()
        self.logits = (torch.randn((tokens, rows), generator=g) * 2).to(BF16).cuda()
        self.e = Z.make_embed(tokens, rows, dim, scale=3.0)
        self.d = Z.make_distill(tokens, rows, k, temperature=2.0, alpha=0.6, scale=0.5)
        self.ews = torch.empty(max(16, Z.zs_embed_workspace_bytes(self.e)), dtype=torch.uint8,
                               device="cuda")
        self.dws = torch.empty(Z.zs_distill_workspace_bytes(self.d), dtype=torch.uint8,
                               device="cuda")
        n = tokens
        self.out = dict(hidden=torch.zeros((n, dim), dtype=BF16, device="cuda"),
                        grad=torch.zeros((rows, dim), dtype=BF16, device="cuda"),
                        loss=torch.zeros(n, device="cuda"), loss2=torch.zeros(n, device="cuda"),
                        lse=torch.zeros((n, 2), device="cuda"),
                        dl=torch.zeros((n, rows), dtype=BF16, device="cuda"),
                        dl2=torch.zeros((n, rows), dtype=BF16, device="cuda"),
                        total=torch.zeros(1, device="cuda"),
                        count=torch.zeros(1, dtype=torch.int64, device="cuda"))

    def run(self, stream=None):
        o, b = self.out, self.b
        Z.embed_lookup(self.e, b.ids, self.table, o["hidden"], stream=stream)
        Z.distill_loss_grad(self.d, self.logits, b.teacher_ids, b.teacher_logits, o["loss"],
                            o["dl"], labels=b.labels, loss_sum=o["total"], counted=o["count"],
                            workspace=self.dws, stream=stream)
        Z.distill_loss(self.d, self.logits, b.teacher_ids, b.teacher_logits, o["loss2"], o["lse"],
                       labels=b.labels, workspace=self.dws, stream=stream)
        Z.distill_grad(self.d, self.logits, b.teacher_ids, b.teacher_logits, o["lse"], o["dl2"],
                       labels=b.labels, stream=stream)
        Z.embed_grad(self.e, b.ids, o["hidden"], o["grad"], self.ews, stream=stream)
        Z.embed_grad(self.e, b.ids, o["hidden"], o["grad"], self.ews, accumulate=True,
                     stream=stream)

    def snapshot(self):
        torch.cuda.synchronize()
        return {k: v.clone() for k, v in self.out.items()}


SHAPES = [(9, 50, 24, 3), (100, 20000, 40, 6), (700, 3000, 72, 5)]


@pytest.mark.parametrize("shape", SHAPES)
def test_captured_calls_replay_equal_eager(shape):
    c = Calls(*shape, seed=5)
    Z.zs_init()
    c.run()
    want = c.snapshot()
    # other inputs in the same buffers, so that a replay must compute
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for k in range(4):
        other = Calls(*shape, seed=6 + k)
        for name in ("ids", "teacher_ids", "teacher_logits", "labels"):
            getattr(c.b, name).copy_(getattr(other.b, name))
        c.logits.copy_(other.logits)
        c.table.copy_(other.table)
        graph.replay()
        got = c.snapshot()
        other.run()
        eager = other.snapshot()
        assert all(torch.equal(got[n], eager[n]) for n in got), f"replay {k}"
        assert not torch.equal(got["dl"], want["dl"])
        assert bool(torch.isfinite(torch.randn(1 << 16, device="cuda").sum()))


def test_capture_first_after_zs_init():
    child = os.path.join(os.path.dirname(os.path.abspath(__file__)), "vocab_capture_child.py")
    r = subprocess.run([sys.executable, "-u", child], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "capture-first ok" in r.stdout, r.stdout[-500:] + r.stderr[-1500:]


def test_streams_and_threads_match_serial():
    serial = []
    for k in range(4):
        c = Calls(*SHAPES[k % 3], seed=20 + k)
        c.run()
        serial.append(c.snapshot())
    calls = [Calls(*SHAPES[k % 3], seed=20 + k) for k in range(4)]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    errors = []

    def work(c, s):
        try:
            for _ in range(5):
                c.run(stream=s)
            s.synchronize()
        except Exception as e:      # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=x) for x in zip(calls, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for c, want in zip(calls, serial):
        got = c.snapshot()
        assert all(torch.equal(got[n], want[n]) for n in got)


def test_half_step_of_the_types():
    assert half_step(BF16) == 2.0 ** -8 and half_step(F32) == U


def test_tensors_of_another_device_are_refused(monkeypatch):
    c = Calls(*SHAPES[0], seed=1)
    c.run()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    o, b = c.out, c.b
    for call in (lambda: Z.embed_lookup(c.e, b.ids, c.table, o["hidden"], stream=0),
                 lambda: Z.embed_grad(c.e, b.ids, o["hidden"], o["grad"], c.ews, stream=0),
                 lambda: Z.distill_loss(c.d, c.logits, b.teacher_ids, b.teacher_logits, o["loss"],
                                        o["lse"], labels=b.labels, workspace=c.dws, stream=0),
                 lambda: Z.distill_grad(c.d, c.logits, b.teacher_ids, b.teacher_logits, o["lse"],
                                        o["dl"], labels=b.labels, stream=0),
                 lambda: Z.distill_loss_grad(c.d, c.logits, b.teacher_ids, b.teacher_logits,
                                             o["loss"], o["dl"], labels=b.labels,
                                             workspace=c.dws, stream=0)):
        with pytest.raises(ValueError, match="current device"):
            call()
