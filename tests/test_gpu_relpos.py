"""The position bias and its gradient against 64-bit forms.

A place of the bias is one fused multiply-add (one fp32 rounding; none for the
bias alone) and one rounding to the output type: u |value|, then half a step.
The table's gradient sums fp32 values: a place goes through at most 8 additions
in its lane, 16 from lane to lane (a tile's rows by 8, or 32 by 4 after 4), 16 of
a bucket's diagonals in a lane or 10 and the wave's 6, 8 groups and 4 waves: fewer
than 64, each of at most u times the sum of absolute values; then fp64, one
rounding to fp32 and one to the type."""
import math

import pytest
import torch

import fsdp_sharded_optimizer_zero_amd as Z
from relpos_util import U, buckets_of, ref_bias, ref_grad

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
KIND = {BF16: Z.ZS_BF16, F32: Z.ZS_F32, torch.int32: Z.ZS_ID_I32, torch.int64: Z.ZS_ID_I64}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def close(name, got, want, err, dtype):
    got, want = got.cpu().double(), want
    fine = torch.isfinite(want)
    assert torch.equal(fine, torch.isfinite(got)), name
    assert torch.equal(got[~fine], want[~fine]), name
    bound = err + half_step(dtype) * (want.abs() + err) + 1e-40
    off = (got - want).abs()
    assert bool((off[fine] <= bound[fine]).all()), (name, float((off / bound)[fine].max()))


def data(r, dtype, seed=0, table=F32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((r.batch, r.heads, r.queries, r.keys), generator=g, device="cuda").to(dtype)
    t = torch.randn((r.buckets, r.heads), generator=g, device="cuda").to(table)
    return x, t


def guarded(shape, dtype):
    n = math.prod(shape)
    buf = torch.full((n + 64,), -7.0, dtype=dtype, device="cuda")
    return buf, buf[32:32 + n].view(shape)


def check(r, dtype, table_dtype=F32, lengths=None, starts=None, seed=0, scores=True, grads=True):
    x, table = data(r, dtype, seed, table_dtype)
    shape = x.shape
    for s in ([None, x] if scores else [None]):
        buf, out = guarded(shape, dtype)
        Z.relpos_bias(r, table, out, scores=s, key_lengths=lengths, query_starts=starts)
        want, size = ref_bias(r, table, s, lengths, starts)
        close("bias", out, want, U * size if s is not None else 0 * size, dtype)
        assert bool((buf[:32] == -7.0).all()) and bool((buf[-32:] == -7.0).all())
    if not grads:
        return
    total, size, ds = ref_grad(r, x, lengths, starts)
    ws = torch.full((Z.zs_relpos_workspace_bytes(r) + 256,), 0xFF, dtype=torch.uint8,
                    device="cuda")
    old = torch.randn((r.buckets, r.heads), device="cuda").to(table_dtype)
    for with_scores in (False, True):
        for acc in (False, True):
            buf, dt = guarded((r.buckets, r.heads), table_dtype)
            dt.copy_(old)
            sbuf, dscores = guarded(shape, dtype)
            src = x.clone()
            Z.relpos_bias_grad(r, src, dt, ws[:-256], dscores if with_scores else None, lengths,
                               starts, accumulate=acc)
            want = total + (old.cpu().double() if acc else 0.0)
            # fp64 from the tiles on, rounded to fp32 first
            close("table", dt, want, 64 * U * size + U * want.abs(), table_dtype)
            assert bool((buf[:32] == -7.0).all()) and bool((buf[-32:] == -7.0).all())
            assert torch.equal(src, x) and bool((ws[-256:] == 0xFF).all())
            assert bool((sbuf[:32] == -7.0).all()) and bool((sbuf[-32:] == -7.0).all())
            if with_scores:
                close("scores", dscores, ds, U * ds.abs(), dtype)
            else:
                assert bool((sbuf == -7.0).all())


SHAPES = [(1, 1, 1, 1), (2, 3, 1, 70), (1, 2, 5, 1), (3, 4, 17, 33), (1, 1, 9, 511), (1, 2, 8, 512),
          (2, 1, 130, 513), (1, 3, 129, 65), (1, 1, 300, 300), (1, 2, 7, 2047), (1, 1, 40, 2049),
          (2, 5, 33, 8), (1, 1, 257, 1030)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype,table,two,causal", [(BF16, F32, True, False), (F32, BF16, True, True),
                                                    (BF16, BF16, False, True),
                                                    (F32, F32, False, False)])
def test_shapes(shape, dtype, table, two, causal):
    b, h, q, k = shape
    r = Z.make_relpos(h, q, k, batch=b, bidirectional=two, causal=causal, dtype=KIND[dtype],
                      table_dtype=KIND[table], scale=0.3)
    check(r, dtype, table, seed=q * k)


BUCKETS = [(2, False, 2), (2, False, 100), (3, False, 5), (4, True, 2), (5, True, 9), (8, True, 3),
           (16, False, 9), (32, True, 128), (32, False, 128), (32, True, 9), (64, False, 64),
           (100, True, 1000), (255, False, 256), (256, False, 129), (256, True, 800),
           (256, True, 65)]


@pytest.mark.parametrize("buckets,two,far", BUCKETS)
def test_buckets(buckets, two, far):
    """Every distance's bucket, the borders among them: a table that holds the
    buckets' numbers."""
    n = min(2 * far, 900) + 10
    r = Z.make_relpos(1, n, n, buckets=buckets, max_distance=far, bidirectional=two,
                      dtype=Z.ZS_F32)
    table = torch.arange(buckets, dtype=F32, device="cuda")[:, None].contiguous()
    out = torch.empty((1, 1, n, n), device="cuda")
    Z.relpos_bias(r, table, out)
    d = torch.arange(n)[None, :] - torch.arange(n)[:, None]
    assert torch.equal(out[0, 0].cpu().long(), buckets_of(r, d))
    check(r, F32, seed=buckets, scores=False)


def test_borders_of_far_distances():
    """Whole borders (powers) far from the origin, through one token's start."""
    for far, buckets in ((1 << 29, 64), (1 << 20, 32), (3 ** 12, 28)):
        r = Z.make_relpos(1, 1, 65, buckets=buckets, max_distance=far, bidirectional=False,
                          dtype=Z.ZS_F32, batch=1)
        from relpos_util import side_bucket
        table = torch.arange(buckets, dtype=F32, device="cuda")[:, None].contiguous()
        out = torch.empty((1, 1, 1, 65), device="cuda")
        exact, m = buckets // 2, buckets - buckets // 2
        for k in range(1, m + 1):
            border = round(exact * (far / exact) ** (k / m))
            r.query_start = min(border + 32, Z.ZS_RELPOS_FAR)
            Z.relpos_bias(r, table, out)
            want = [side_bucket(max(r.query_start - j, 0), buckets, far) for j in range(65)]
            assert out.reshape(-1).tolist() == want


@pytest.mark.parametrize("start", [-400, -30, 0, 5, 700, 100000, Z.ZS_RELPOS_FAR,
                                   -Z.ZS_RELPOS_FAR])
@pytest.mark.parametrize("causal", [False, True])
def test_starts(start, causal):
    r = Z.make_relpos(3, 70, 300, batch=2, query_start=start, causal=causal, dtype=Z.ZS_BF16)
    check(r, BF16)


@pytest.mark.parametrize("ids", [torch.int32, torch.int64])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("queries", [1, 40])
def test_lengths_and_starts(ids, causal, queries):
    """A padded batch and one token a sequence: lengths of 0, 1, all, and beyond
    the range they are held to; positions of their own."""
    keys = 261
    lengths = torch.tensor([0, 1, 37, keys, keys + 9, -3], dtype=ids)
    starts = torch.tensor([0, 0, 36, keys - 1, 100, -50], dtype=ids)
    r = Z.make_relpos(5, queries, keys, batch=6, bidirectional=False, causal=causal, scale=0.125,
                      dtype=Z.ZS_F32, id_dtype=KIND[ids])
    for ln, st in ((lengths, None), (None, starts), (lengths, starts)):
        check(r, F32, lengths=None if ln is None else ln.cuda(),
              starts=None if st is None else st.cuda(), seed=3)


def test_starts_past_the_range_are_held_to_it():
    far = Z.ZS_RELPOS_FAR
    r = Z.make_relpos(1, 2, 70, batch=3, dtype=Z.ZS_F32, id_dtype=Z.ZS_ID_I64)
    _, table = data(r, F32)
    out = torch.empty((3, 1, 2, 70), device="cuda")
    Z.relpos_bias(r, table, out,
                  query_starts=torch.tensor([1 << 62, -(1 << 62), far], device="cuda"))
    assert bool((out[0] == table[15]).all()) and bool((out[1] == table[31]).all())
    assert torch.equal(out[0], out[2])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, "lowest"])
def test_what_is_masked_is_not_read(dtype, bad):
    """Values of any kind in places that are not seen change nothing; in places
    that are seen they propagate."""
    bad = torch.finfo(dtype).min if bad == "lowest" else bad
    r = Z.make_relpos(3, 50, 90, batch=2, causal=True, query_start=20, dtype=KIND[dtype],
                      bidirectional=False)
    lengths = torch.tensor([60, 33], device="cuda")
    x, table = data(r, dtype)
    i = torch.arange(50, device="cuda")[:, None] + 20
    j = torch.arange(90, device="cuda")[None, :]
    seen = ((j <= i)[None] & (j < lengths[:, None, None]))[:, None].expand_as(x)
    y = torch.where(seen, x, bad)
    outs = [torch.empty_like(x) for _ in range(2)]
    for s, o in zip((x, y), outs):
        Z.relpos_bias(r, table, o, scores=s, key_lengths=lengths)
    assert torch.equal(*outs) and bool((outs[0][~seen] == -math.inf).all())
    assert bool(torch.isfinite(outs[0][seen]).all())
    ws = torch.empty(Z.zs_relpos_workspace_bytes(r), dtype=torch.uint8, device="cuda")
    grads = [(torch.empty((32, 3), device="cuda"), torch.empty_like(x)) for _ in range(2)]
    for s, (dt, ds) in zip((x, y), grads):
        Z.relpos_bias_grad(r, s, dt, ws, ds, key_lengths=lengths)
    assert torch.equal(grads[0][0], grads[1][0]) and torch.equal(grads[0][1], grads[1][1])
    assert bool((grads[1][1][~seen] == 0).all())
    if bad != bad:
        y[0, 1, 40, 5] = bad                        # seen: head 1 alone is NaN there
        Z.relpos_bias_grad(r, y, grads[1][0], ws, key_lengths=lengths)
        assert int(torch.isnan(grads[1][0]).sum()) == 1
        Z.relpos_bias(r, table, outs[1], scores=y, key_lengths=lengths)
        assert int(torch.isnan(outs[1]).sum()) == 1


PITCHES = ["by_query", "padded", "offset"]


@pytest.mark.parametrize("how", PITCHES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides(how, dtype):
    b, h, q, k = 2, 3, 37, 203
    if how == "by_query":
        make = lambda: torch.full((b, q, h, k), -7.0, dtype=dtype, device="cuda").transpose(1, 2)
    elif how == "padded":
        make = lambda: torch.full((b, h, q, k + 5), -7.0, dtype=dtype, device="cuda")[..., :k]
    else:
        make = lambda: torch.full((b, h + 1, q, k), -7.0, dtype=dtype, device="cuda")[:, 1:]
    x, out = make(), make()
    pitch = x.stride()[:3]
    r = Z.make_relpos(h, q, k, batch=b, in_pitch=pitch, out_pitch=pitch, dtype=KIND[dtype],
                      scale=0.5, table_pitch=7)
    full, _ = data(r, dtype, 4)
    x.copy_(full)
    wide = torch.randn((32, 7), device="cuda")
    table = wide[:, :h]
    lengths = torch.tensor([k, 100], device="cuda")
    want, size = ref_bias(r, table, full, lengths, None)
    Z.relpos_bias(r, table, out, scores=x, key_lengths=lengths)
    close("bias", out, want, U * size, dtype)
    base = out._base.clone()
    out.fill_(-7.0)
    assert bool((out._base == -7.0).all()), "written outside the places"
    total, size, ds = ref_grad(r, full, lengths, None)
    ws = torch.empty(Z.zs_relpos_workspace_bytes(r), dtype=torch.uint8, device="cuda")
    grad_wide = torch.full((32, 7), -7.0, device="cuda")
    Z.relpos_bias_grad(r, x, grad_wide[:, :h], ws, out, key_lengths=lengths)
    close("table", grad_wide[:, :h], total, 64 * U * size + U * total.abs(), F32)
    assert bool((grad_wide[:, h:] == -7.0).all())
    close("scores", out, ds, U * ds.abs(), dtype)
    # in place
    y = make()
    y.copy_(full)
    Z.relpos_bias(r, table, y, scores=y, key_lengths=lengths)
    assert torch.equal(y._base, base)
    y.copy_(full)
    again = torch.empty((32, 7), device="cuda")
    Z.relpos_bias_grad(r, y, again[:, :h], ws, y, key_lengths=lengths)
    assert torch.equal(again[:, :h], grad_wide[:, :h]) and torch.equal(y, out)


@pytest.mark.parametrize("empty", [dict(batch=0), dict(queries=0), dict(keys=0)])
def test_nothing_there(empty):
    sizes = dict(batch=2, queries=5, keys=6) | empty
    r = Z.make_relpos(3, sizes["queries"], sizes["keys"], batch=sizes["batch"])
    x = torch.empty((sizes["batch"], 3, sizes["queries"], sizes["keys"]), dtype=BF16,
                    device="cuda")
    table = torch.ones((32, 3), device="cuda")
    ws = torch.empty(Z.zs_relpos_workspace_bytes(r), dtype=torch.uint8, device="cuda")
    Z.relpos_bias(r, table, x)
    Z.relpos_bias_grad(r, x, table, ws, accumulate=True)
    assert bool((table == 1).all())
    Z.relpos_bias_grad(r, x, table, ws)
    assert bool((table == 0).all())


def test_past_32_bits():
    """More than 2^31 places; the last heads and rows are looked at."""
    h, q, k = 33, 8192, 8200
    r = Z.make_relpos(h, q, k, dtype=Z.ZS_BF16)
    table = torch.randn((32, h), device="cuda")
    out = torch.empty((1, h, q, k), dtype=BF16, device="cuda")
    Z.relpos_bias(r, table, out)
    d = torch.arange(k)[None, :] - torch.arange(q - 3, q)[:, None]
    want = table.cpu()[buckets_of(r, d)].permute(2, 0, 1).to(BF16)
    assert torch.equal(out[0, :, q - 3:].cpu(), want)
    out.zero_()
    out[0, -1, -1, -1] = 5.0        # d = 8: two-sided bucket 16 + 8
    out[0, -1, -1, 0] = 7.0         # far behind
    out[0, 0, 0, 0] = 3.0
    ws = torch.empty(Z.zs_relpos_workspace_bytes(r), dtype=torch.uint8, device="cuda")
    Z.relpos_bias_grad(r, out, table, ws)
    want = torch.zeros((32, h))
    want[24, -1], want[15, -1], want[0, 0] = 5.0, 7.0, 3.0
    assert torch.equal(table.cpu(), want)


def test_differences():
    """The gradient against differences of the bias in a weighted sum."""
    r = Z.make_relpos(2, 30, 41, batch=2, causal=True, query_start=7, scale=0.25, dtype=Z.ZS_F32)
    lengths = torch.tensor([41, 20], device="cuda")
    x, table = data(r, F32, 6)
    g = torch.randn_like(x)

    def value(table, x):
        out = torch.empty_like(x)
        Z.relpos_bias(r, table, out, scores=x, key_lengths=lengths)
        return float((torch.where(torch.isinf(out), 0.0, out).double() * g.double()).sum())

    ws = torch.empty(Z.zs_relpos_workspace_bytes(r), dtype=torch.uint8, device="cuda")
    dt, ds = torch.empty_like(table), torch.empty_like(x)
    Z.relpos_bias_grad(r, g, dt, ws, ds, key_lengths=lengths)
    # the value is linear and all other places cancel: a difference is off by the
    # roundings (2^-22 at values up to 8) of the places of one bucket and head, at
    # most some 600, twice, over the step of 1/4: 1.2e-3 for weights of size 1
    for u in range(32):
        up, down = table.clone(), table.clone()
        up[u, 1] += 0.125
        down[u, 1] -= 0.125
        assert abs((value(up, x) - value(down, x)) / 0.25 - float(dt[u, 1])) < 5e-3
    for at in ((0, 0, 0, 0), (1, 1, 20, 19), (0, 1, 29, 36), (1, 0, 3, 30)):
        up, down = x.clone(), x.clone()
        up[at] += 0.5
        down[at] -= 0.5
        assert abs(value(table, up) - value(table, down) - float(ds[at])) < 5e-3


def test_same_bits_every_time_and_captured():
    """Run to run the same bits; captured with two calls sharing a workspace one
    after the other, replayed over new values with eager calls between."""
    Z.zs_init()
    r = Z.make_relpos(6, 300, 520, batch=3, dtype=Z.ZS_BF16)
    x, table = data(r, BF16, 8)
    x2 = x.flip(3).contiguous()
    ws = torch.empty(Z.zs_relpos_workspace_bytes(r), dtype=torch.uint8, device="cuda")
    dts = [torch.empty((32, 6), device="cuda") for _ in range(2)]
    out = torch.empty_like(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Z.relpos_bias(r, table, out, scores=x)
        Z.relpos_bias_grad(r, x, dts[0], ws)
        Z.relpos_bias_grad(r, x2, dts[1], ws)
    for k in range(4):
        x.copy_(data(r, BF16, 40 + k)[0])
        x2.copy_(x.flip(3))
        graph.replay()
        torch.cuda.synchronize()
        eager = [torch.empty_like(d) for d in dts]
        eout = torch.empty_like(out)
        Z.relpos_bias(r, table, eout, scores=x)
        ws2 = torch.full_like(ws, 0xFF)
        for e, s in zip(eager, (x, x2)):
            Z.relpos_bias_grad(r, s, e, ws2)
        assert all(torch.equal(a, b) for a, b in zip(dts, eager)) and torch.equal(out, eout)


def test_streams():
    """Calls on two streams at once, each with its own workspace."""
    r = Z.make_relpos(4, 200, 300, batch=2, dtype=Z.ZS_F32)
    streams = [torch.cuda.Stream() for _ in range(2)]
    xs = [data(r, F32, 50 + k)[0] for k in range(2)]
    want = [ref_grad(r, x, None, None) for x in xs]
    ws = [torch.empty(Z.zs_relpos_workspace_bytes(r), dtype=torch.uint8, device="cuda")
          for _ in range(2)]
    dts = [torch.empty((32, 4), device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, x, d, w in zip(streams, xs, dts, ws):
            Z.relpos_bias_grad(r, x, d, w, stream=st)
    torch.cuda.synchronize()
    for d, (total, size, _) in zip(dts, want):
        close("table", d, total, 64 * U * size + U * total.abs(), F32)


def test_small_grid_build():
    """At most 256 blocks a launch."""
    with Z.library(Z.SMALLGRID_LIB_PATH):
        r = Z.make_relpos(12, 200, 90, batch=9, dtype=Z.ZS_F32, causal=True)
        check(r, F32)
        check(Z.make_relpos(7, 1, 3000, batch=64, bidirectional=False, dtype=Z.ZS_BF16), BF16)


def test_binding_refuses():
    r = Z.make_relpos(4, 10, 20, batch=3)
    x, table = data(r, BF16)
    with pytest.raises(ValueError, match="the call needs"):
        Z.relpos_bias(r, table, x.transpose(2, 3))
    with pytest.raises(ValueError, match="key_lengths"):
        Z.relpos_bias(r, table, x, key_lengths=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="GPU tensor"):
        Z.relpos_bias(r, table, x, key_lengths=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="table"):
        Z.relpos_bias(r, table.to(BF16), x)
    with pytest.raises(Z.ZSError, match="workspace"):
        Z.relpos_bias_grad(r, x, table, torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="workspace"):
        Z.relpos_bias_grad(r, x, table, torch.empty(16, dtype=torch.uint8, device="cuda"),
                           workspace_bytes=4096)


def test_tensors_of_another_device_are_refused(monkeypatch):
    r = Z.make_relpos(4, 10, 20, batch=3, dtype=Z.ZS_F32)
    x, table = data(r, F32)
    ws = torch.empty(Z.zs_relpos_workspace_bytes(r), dtype=torch.uint8, device="cuda")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in (lambda: Z.relpos_bias(r, table, x, stream=0),
                 lambda: Z.relpos_bias_grad(r, x, table, ws, stream=0)):
        with pytest.raises(ValueError, match="current device"):
            call()


@pytest.mark.parametrize("keys", [1, 3, 5, 7, 8, 9, 15, 512 + 7, 1024 + 1, 4096 + 3])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_ends_of_rows(keys, dtype):
    """Rows of fewer keys than a vector, and every way a row can end in one,
    the last row's end being the tensor's; in place too."""
    r = Z.make_relpos(2, 13, keys, batch=2, dtype=KIND[dtype], query_start=keys // 2, scale=0.5)
    lengths = torch.tensor([keys, max(1, keys - 1)], device="cuda")
    check(r, dtype, lengths=lengths, seed=keys)
    x, table = data(r, dtype, keys)
    want = torch.empty_like(x)
    Z.relpos_bias(r, table, want, scores=x, key_lengths=lengths)
    y = x.clone()
    Z.relpos_bias(r, table, y, scores=y, key_lengths=lengths)
    assert torch.equal(y, want)
    ws = torch.empty(Z.zs_relpos_workspace_bytes(r), dtype=torch.uint8, device="cuda")
    dt, dx = torch.empty_like(table), torch.empty_like(x)
    Z.relpos_bias_grad(r, x, dt, ws, dx, key_lengths=lengths)
    y, again = x.clone(), torch.empty_like(table)
    Z.relpos_bias_grad(r, y, again, ws, y, key_lengths=lengths)
    assert torch.equal(y, dx) and torch.equal(dt, again)


def test_many_rows_and_sequences():
    """More tiles than the GPU holds at once, in stretches and at their end."""
    r = Z.make_relpos(16, 100, 70, batch=70, dtype=Z.ZS_BF16, causal=True)
    check(r, BF16, seed=1)
    r = Z.make_relpos(33, 1, 2100, batch=65, dtype=Z.ZS_BF16, bidirectional=False, scale=0.125)
    starts = torch.randint(0, 2100, (65,), generator=torch.Generator().manual_seed(1))
    check(r, BF16, lengths=(starts + 1).cuda(), starts=starts.cuda(), seed=2)


@pytest.mark.parametrize("start", [Z.ZS_RELPOS_FAR, -Z.ZS_RELPOS_FAR])
@pytest.mark.parametrize("by_query", [True, False])
def test_ends_of_the_range(start, by_query):
    """As many queries, or keys, as a call may have, at the ends of the positions:
    a gradient of ones counts the places of each bucket, and the bias of the
    first and last places is their bucket's."""
    far = Z.ZS_RELPOS_FAR
    q, k = (far, 1) if by_query else (1, far)
    r = Z.make_relpos(1, q, k, query_start=start, dtype=Z.ZS_BF16)
    g = torch.ones((1, 1, q, k), dtype=BF16, device="cuda")
    ws = torch.empty(Z.zs_relpos_workspace_bytes(r), dtype=torch.uint8, device="cuda")
    dt = torch.empty((32, 1), device="cuda")
    Z.relpos_bias_grad(r, g, dt, ws)
    # distances run over a stretch of far numbers from d0 on
    d0 = (-start - (far - 1)) if by_query else -start
    first = max(d0, -200)
    near = torch.arange(first, max(first, min(d0 + far, 200)))
    want = torch.bincount(buckets_of(r, near), minlength=32).double() if len(near) else \
        torch.zeros(32, dtype=torch.float64)
    want[15] += max(0, min(d0 + far, -200) - d0)
    want[31] += max(0, d0 + far - max(d0, 200))
    # counts of up to 2^29: exact in the tiles and in fp64, rounded once to fp32
    assert want.sum() == far and torch.equal(dt[:, 0].cpu(), want.float())
    table = torch.arange(32, dtype=F32, device="cuda")[:, None].contiguous()
    Z.relpos_bias(r, table, g)
    flat = g.reshape(-1)
    at = torch.tensor([0, 1, 130, far // 2, far - 131, far - 2, far - 1])
    d = (-at - start) if by_query else (at - start)
    assert torch.equal(flat[at.cuda()].cpu().long(), buckets_of(r, d))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("causal", [False, True])
def test_scores_past_the_caches(dtype, causal):
    """Calls large enough for loads past the caches' reuse, rows of an odd length,
    against one call a sequence, which are not; in place too.  A place's bias and
    its scores' gradient do not depend on how a call is cut; gradients of -1, 0
    and 1 are summed exactly in any order (2.1 million places a plane, 10.6 million
    a head: below 2^24)."""
    b, h, q, k = 5, 8, 1031, 2053
    kw = dict(dtype=KIND[dtype], causal=causal, query_start=900 if causal else 0, scale=0.5,
              bidirectional=not causal)
    r, one = Z.make_relpos(h, q, k, batch=b, **kw), Z.make_relpos(h, q, k, **kw)
    limit = 160 << 20
    assert h * q * k * (2 if dtype == BF16 else 4) < limit <= b * h * q * k * 2
    x, table = data(r, dtype, 11)
    lengths = torch.tensor([k, 2048, 700, 0, 1], device="cuda")
    want = torch.empty_like(x)
    for i in range(b):
        Z.relpos_bias(one, table, want[i:i + 1], scores=x[i:i + 1], key_lengths=lengths[i:i + 1])
    out = torch.empty_like(x)
    Z.relpos_bias(r, table, out, scores=x, key_lengths=lengths)
    assert torch.equal(out, want)
    out.copy_(x)
    Z.relpos_bias(r, table, out, scores=out, key_lengths=lengths)
    assert torch.equal(out, want)
    g = torch.Generator(device="cuda").manual_seed(12)
    x = torch.randint(-1, 2, x.shape, generator=g, device="cuda", dtype=torch.int8).to(dtype)
    ws = torch.empty(Z.zs_relpos_workspace_bytes(r), dtype=torch.uint8, device="cuda")
    dt = torch.zeros((32, h), device="cuda")
    for i in range(b):
        Z.relpos_bias_grad(one, x[i:i + 1], dt, ws, want[i:i + 1], lengths[i:i + 1],
                           accumulate=True)
    assert bool((dt != 0).any()) and float(dt.abs().max()) < 2.0 ** 24
    for place in (None, out, x):
        got = torch.full_like(dt, math.nan)
        Z.relpos_bias_grad(r, x, got, ws, place, lengths)
        assert torch.equal(got, dt)
        if place is not None:
            assert torch.equal(place, want)


@pytest.mark.parametrize("dtype,keys", [(BF16, 82003), (F32, 41001)])
def test_one_token_a_sequence_past_the_caches(dtype, keys):
    """The same for one query, four vectors a lane."""
    b, h = 64, 16
    kw = dict(dtype=KIND[dtype], scale=0.5, bidirectional=False, causal=True)
    r, one = Z.make_relpos(h, 1, keys, batch=b, **kw), Z.make_relpos(h, 1, keys, **kw)
    x, table = data(r, dtype, 13)
    assert x.numel() * x.element_size() >= 160 << 20
    starts = torch.randint(0, keys, (b,), generator=torch.Generator().manual_seed(14)).cuda()
    starts[0], starts[1] = 0, keys - 1
    lengths = starts + 1
    want, out = torch.empty_like(x), torch.empty_like(x)
    for i in range(b):
        Z.relpos_bias(one, table, want[i:i + 1], scores=x[i:i + 1], key_lengths=lengths[i:i + 1],
                      query_starts=starts[i:i + 1])
    Z.relpos_bias(r, table, out, scores=x, key_lengths=lengths, query_starts=starts)
    assert torch.equal(out, want)
    Z.relpos_bias(r, table, x, scores=x, key_lengths=lengths, query_starts=starts)
    assert torch.equal(x, want)


def test_one_token_a_sequence_fp32():
    """Four vectors a lane in fp32 (more than 8192 tiles), onto scores and alone."""
    r = Z.make_relpos(33, 1, 2101, batch=65, dtype=Z.ZS_F32, bidirectional=False, scale=0.125)
    starts = torch.randint(0, 2101, (65,), generator=torch.Generator().manual_seed(1))
    lengths, starts = (starts + 1).cuda(), starts.cuda()
    check(r, F32, lengths=lengths, starts=starts, seed=2, grads=False)
    x, table = data(r, F32, 2)
    want = torch.empty_like(x)
    Z.relpos_bias(r, table, want, scores=x, key_lengths=lengths, query_starts=starts)
    Z.relpos_bias(r, table, x, scores=x, key_lengths=lengths, query_starts=starts)
    assert torch.equal(x, want)
