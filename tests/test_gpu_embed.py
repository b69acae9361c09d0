"""Embedding lookup and gradient on the GPU against plain 64-bit forms."""
import math

import pytest
import torch

import fsdp_sharded_optimizer_zero_amd as Z
from vocab_util import (KIND, U, assert_guards, embed_grad_bound, guarded, half_step,
                        ref_embed_grad, ref_lookup)

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def make_ids(kind, n, vocab, seed, dtype=torch.int64):
    g = torch.Generator().manual_seed(seed)
    if kind == "zipf":
        u = torch.rand(n, generator=g, dtype=torch.float64)
        ids = (torch.exp(u * math.log(vocab + 1.0)) - 1).long().clamp(0, vocab - 1)
    elif kind == "uniform":
        ids = torch.randint(0, vocab, (n,), generator=g)
    elif kind == "one":
        ids = torch.full((n,), vocab // 2)
    elif kind == "two":                      # two long runs, interleaved
        ids = torch.arange(n) % 2 * (vocab - 1)
    elif kind == "descending":
        ids = (vocab - 1 - torch.arange(n)) % vocab
    else:                                    # none in range
        ids = torch.where(torch.arange(n) % 2 == 0, -1 - torch.arange(n), vocab + torch.arange(n))
    return ids.to(dtype).cuda()


def values(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).cuda()


# ---- lookup ------------------------------------------------------------------------

@pytest.mark.parametrize("table_dtype", [BF16, F32])
@pytest.mark.parametrize("act_dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,rows,dim,pad", [(1, 1, 1, 0), (1, 1000, 4096, 0), (3, 7, 9, 0),
                                                 (257, 50, 64, 8), (100, 333, 771, 5),
                                                 (17, 20, 8200, 1), (0, 4, 8, 0)])
def test_lookup(table_dtype, act_dtype, tokens, rows, dim, pad):
    first, scale = 5, 1.5
    ids = make_ids("uniform", tokens, rows + 10, 1, torch.int32)   # some before, some behind
    tbuf, table = guarded(rows, dim, dim + pad, table_dtype, float("nan"))
    table.copy_(values((rows, dim), table_dtype, 2))
    obuf, out = guarded(tokens, dim, dim + 2 * pad, act_dtype)
    e = Z.make_embed(tokens, rows, dim, first_row=first, table_pitch=dim + pad,
                     act_pitch=dim + 2 * pad, id_dtype=Z.ZS_ID_I32, table_dtype=KIND[table_dtype],
                     act_dtype=KIND[act_dtype], scale=scale)
    Z.embed_lookup(e, ids, table, out)
    torch.cuda.synchronize()
    want = ref_lookup(ids, table, first, scale)
    # one fp32 product, one rounding to the output
    off = (out.cpu().double() - want).abs()
    assert bool((off <= want.abs() * (half_step(act_dtype) * (1 + U) + U)).all())
    assert_guards(obuf, tokens, dim, dim + 2 * pad)


def test_lookup_values_pass_through():
    """Scale 1 copies every finite and infinite value; NaN stays NaN; a row
    that is not here is +0 even where the scale is negative."""
    table = torch.tensor([[0.0, -0.0, math.inf, -math.inf, math.nan, 1e-40, 3.4e38, -1.0]]).cuda()
    ids = torch.tensor([0, -1, 1], dtype=torch.int64).cuda()
    out = torch.full((3, 8), 9.0, device="cuda")
    Z.embed_lookup(Z.make_embed(3, 1, 8, table_dtype=Z.ZS_F32, act_dtype=Z.ZS_F32), ids, table, out)
    assert torch.equal(out[0].nan_to_num(nan=5.0), table[0].nan_to_num(nan=5.0))
    assert bool((out[1:].view(torch.int32) == 0).all())
    Z.embed_lookup(Z.make_embed(3, 1, 8, table_dtype=Z.ZS_F32, act_dtype=Z.ZS_F32, scale=-2.0),
                   ids, table, out)
    assert bool((out[1:].view(torch.int32) == 0).all())


def test_every_bf16_rounding():
    """fp32 -> bf16 at every kept half (subnormals, infinities, NaN) and the
    dropped halves around the middle: torch's CPU cast, NaN as a class."""
    hi = torch.arange(1 << 16, dtype=torch.int64) << 16
    low = torch.tensor([0, 1, 0x7FFF, 0x8000, 0x8001, 0xFFFF])
    bits = (hi[:, None] | low).to(torch.int64)
    bits = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32).flatten()
    x = bits.view(F32).reshape(-1, 1024)
    n = x.shape[0]
    out = torch.empty((n, 1024), dtype=BF16, device="cuda")
    e = Z.make_embed(n, n, 1024, table_dtype=Z.ZS_F32)
    Z.embed_lookup(e, torch.arange(n).cuda(), x.cuda(), out)
    want, got = x.to(BF16), out.cpu()
    nan = torch.isnan(x)
    assert bool((torch.isnan(got) == nan).all())
    assert torch.equal(got.view(torch.int16)[~nan], want.view(torch.int16)[~nan])


def test_extreme_ids_are_not_here():
    lim = torch.iinfo(torch.int64)
    ids = torch.tensor([lim.min, lim.max, -1, 10, 14, 2 ** 32 + 10, lim.min + 10]).cuda()
    table = values((4, 16), F32, 3)
    out = torch.full((7, 16), 9.0, device="cuda")
    e = Z.make_embed(7, 4, 16, first_row=10, table_dtype=Z.ZS_F32, act_dtype=Z.ZS_F32)
    Z.embed_lookup(e, ids, table, out)
    assert torch.equal(out[3], table[0])
    assert bool((out[[0, 1, 2, 4, 5, 6]] == 0).all())
    grad = torch.full((4, 16), 9.0, device="cuda")
    ws = torch.empty(Z.zs_embed_workspace_bytes(e), dtype=torch.uint8, device="cuda")
    act = values((7, 16), F32, 4)
    Z.embed_grad(e, ids, act, grad, ws)
    assert torch.equal(grad[0], act[3]) and bool((grad[1:] == 0).all())


def test_table_and_offsets_past_32_bits():
    """Element offsets above 2^32 in the table, the activations and the gradient."""
    rows, dim = 3, 40
    pitch = (1 << 31) + 72                       # the last row begins past 2^32 elements
    table = torch.empty(2 * pitch + dim, dtype=BF16, device="cuda")
    view = table.as_strided((rows, dim), (pitch, 1))
    view.copy_(values((rows, dim), BF16, 5))
    ids = torch.tensor([2, 0, 1, 2], dtype=torch.int64).cuda()
    out = torch.empty((4, dim), dtype=BF16, device="cuda")
    e = Z.make_embed(4, rows, dim, table_pitch=pitch)
    Z.embed_lookup(e, ids, table, out)
    assert torch.equal(out, view[ids])
    ws = torch.empty(Z.zs_embed_workspace_bytes(e), dtype=torch.uint8, device="cuda")
    act = values((4, dim), BF16, 6)
    Z.embed_grad(e, ids, act, table, ws)
    want, size, count = ref_embed_grad(ids, act, rows, 0, 1.0)
    off = (view.cpu().double() - want).abs()
    assert bool((off <= embed_grad_bound(want, size, count, None, BF16)).all())


# ---- gradient ----------------------------------------------------------------------

def run_grad(ids, tokens, rows, dim, act_dtype, table_dtype, accumulate, first=0, scale=1.0,
             pad=0, seed=7):
    act_buf, act = guarded(tokens, dim, dim + pad, act_dtype, float("nan"))
    act.copy_(values((tokens, dim), act_dtype, seed))
    gbuf, grad = guarded(rows, dim, dim + 3 * pad, table_dtype)
    old = None
    if accumulate:
        grad.copy_(values((rows, dim), table_dtype, seed + 1))
        old = grad.cpu().double()
    e = Z.make_embed(tokens, rows, dim, first_row=first, table_pitch=dim + 3 * pad,
                     act_pitch=dim + pad, id_dtype=KIND[ids.dtype], table_dtype=KIND[table_dtype],
                     act_dtype=KIND[act_dtype], scale=scale)
    need = Z.zs_embed_workspace_bytes(e)
    ws = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    before = grad.clone()
    Z.embed_grad(e, ids, act, grad, ws, accumulate=accumulate, workspace_bytes=need)
    torch.cuda.synchronize()
    assert bool((ws[need:] == 0xA5).all()), "written behind the workspace"
    assert_guards(gbuf, rows, dim, dim + 3 * pad)
    want, size, count = ref_embed_grad(ids, act, rows, first, scale)
    result = want if old is None else want + old
    off = (grad.cpu().double() - result).abs()
    assert bool((off <= embed_grad_bound(want, size, count, old, table_dtype)).all())
    empty = (count == 0).cuda()
    if accumulate:
        assert torch.equal(grad[empty], before[empty]), "a row without tokens changed"
    else:
        assert bool((grad[empty].abs() == 0).all())
    # the same bits again, whatever the workspace held
    again = before.clone() if accumulate else torch.full_like(before, 3.0)
    e2 = Z.make_embed(tokens, rows, dim, first_row=first, act_pitch=dim + pad,
                      id_dtype=KIND[ids.dtype], table_dtype=KIND[table_dtype],
                      act_dtype=KIND[act_dtype], scale=scale)
    again = again.contiguous()
    ws.fill_(0x3C)
    Z.embed_grad(e2, ids, act, again, ws, accumulate=accumulate)
    assert torch.equal(again, grad), "not deterministic"


@pytest.mark.parametrize("kind", ["zipf", "uniform", "one", "two", "descending", "none"])
@pytest.mark.parametrize("tokens,rows,dim", [(1, 1, 1), (7, 5, 3), (9, 300, 64), (65, 50257, 96),
                                             (1025, 255, 130), (4099, 1000, 771)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_grad_orders(kind, tokens, rows, dim, accumulate):
    run_grad(make_ids(kind, tokens, rows, 11), tokens, rows, dim, BF16, F32, accumulate)


@pytest.mark.parametrize("act_dtype", [BF16, F32])
@pytest.mark.parametrize("table_dtype", [BF16, F32])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("tokens", [64, 65, 2051])
def test_grad_types_pitches_ranges(act_dtype, table_dtype, accumulate, pad, tokens):
    ids = make_ids("zipf", tokens, 900, 12, torch.int32)
    run_grad(ids, tokens, 257, 519, act_dtype, table_dtype, accumulate, first=3, scale=22.5,
             pad=pad)


@pytest.mark.parametrize("tokens,rows,dim", [(30011, 700, 72), (70001, 260, 40), (5000, 260000, 24),
                                             (300, 8, 8300), (20000, 1, 256)])
def test_grad_long_runs_and_many_rows(tokens, rows, dim):
    run_grad(make_ids("zipf", tokens, rows, 13), tokens, rows, dim, BF16, F32, False)


WIDTHS = [*range(1, 18), 255, 257, 263, 511, 513, 519, 1025, 1031, 2047, 2049, 2055, 4097]


@pytest.mark.parametrize("act_dtype", [BF16, F32])
@pytest.mark.parametrize("table_dtype", [BF16, F32])
def test_every_end_of_a_row(act_dtype, table_dtype):
    """Rows that end at any place of a vector, at any alignment."""
    for dim in WIDTHS:
        test_lookup(table_dtype, act_dtype, 66, 40, dim, 1)
        for accumulate in (False, True):
            run_grad(make_ids("zipf", 200, 40, 14), 200, 30, dim, act_dtype, table_dtype,
                     accumulate, first=2, scale=-0.5, pad=1)


@pytest.mark.parametrize("kind,tokens,rows", [("one", 40000, 130000), ("two", 40000, 500),
                                              ("runs", 70000, 131072)])
def test_grad_sort_lists_overflow(kind, tokens, rows):
    """More tokens of one sort bucket than its waves list."""
    ids = make_ids("zipf" if kind == "runs" else kind, tokens, rows, 21)
    if kind == "runs":
        ids[1000:9000], ids[30000:52000] = 77, 512
    run_grad(ids, tokens, rows, 24, BF16, F32, False)


def test_grad_many_tokens():
    """A million tokens into a quarter of a million rows, against torch's own
    64-bit index_add on the GPU."""
    tokens, rows, dim = 1 << 20, 1 << 18, 8
    g = torch.Generator(device="cuda").manual_seed(5)
    ids = torch.randint(-5, rows + 5, (tokens,), generator=g, device="cuda")
    ids[::16] = 77
    act = torch.randn((tokens, dim), generator=g, device="cuda")
    e = Z.make_embed(tokens, rows, dim, table_dtype=Z.ZS_F32, act_dtype=Z.ZS_F32)
    ws = torch.empty(Z.zs_embed_workspace_bytes(e), dtype=torch.uint8, device="cuda")
    grad = torch.full((rows, dim), 3.0, device="cuda")
    Z.embed_grad(e, ids, act, grad, ws)
    here = (ids >= 0) & (ids < rows)
    want, size = (torch.zeros((rows, dim), dtype=torch.float64, device="cuda") for _ in range(2))
    want.index_add_(0, ids[here], act[here].double())
    size.index_add_(0, ids[here], act[here].double().abs())
    count = torch.bincount(ids[here], minlength=rows)
    off = (grad.double() - want).abs()
    assert bool((off <= embed_grad_bound(want, size, count, None, F32)).all())


def test_grad_without_tokens():
    e = Z.make_embed(0, 33, 20, table_dtype=Z.ZS_F32)
    ws = torch.empty(max(Z.zs_embed_workspace_bytes(e), 16), dtype=torch.uint8, device="cuda")
    grad = torch.full((33, 20), 4.0, device="cuda")
    ids = torch.empty(0, dtype=torch.int64, device="cuda")
    act = torch.empty((0, 20), dtype=BF16, device="cuda")
    Z.embed_grad(e, ids, act, grad, ws, accumulate=True)
    assert bool((grad == 4.0).all())
    Z.embed_grad(e, ids, act, grad, ws)
    assert bool((grad == 0.0).all())


def test_grad_nan_stays_in_its_row():
    """NaN and infinities of tokens that are not here are not read into any
    sum; those of a token that is reach its own row alone."""
    ids = torch.tensor([2, -1, 0, 2, 9, 1], dtype=torch.int64).cuda()
    act = values((6, 12), F32, 14)
    act[1], act[4], act[5, 3] = math.nan, math.inf, math.nan
    e = Z.make_embed(6, 4, 12, table_dtype=Z.ZS_F32, act_dtype=Z.ZS_F32)
    ws = torch.empty(Z.zs_embed_workspace_bytes(e), dtype=torch.uint8, device="cuda")
    grad = torch.full((4, 12), 3.0, device="cuda")
    Z.embed_grad(e, ids, act, grad, ws)
    nan = torch.isnan(grad)
    assert int(nan.sum()) == 1 and bool(nan[1, 3])
    assert torch.equal(grad[2], act[0] + act[3]) and bool((grad[3] == 0).all())


def test_grad_matches_differences():
    """The gradient of f(W) = <lookup(W), A> by central differences (f is
    linear in W, so they are exact up to rounding)."""
    rows, dim, tokens, scale = 5, 6, 9, 3.0
    ids = make_ids("uniform", tokens, rows, 15)
    act = values((tokens, dim), F32, 16)
    table = values((rows, dim), F32, 17)
    e = Z.make_embed(tokens, rows, dim, table_dtype=Z.ZS_F32, act_dtype=Z.ZS_F32, scale=scale)
    ws = torch.empty(Z.zs_embed_workspace_bytes(e), dtype=torch.uint8, device="cuda")
    grad = torch.empty((rows, dim), device="cuda")
    Z.embed_grad(e, ids, act, grad, ws)

    def f(w):
        out = torch.empty((tokens, dim), device="cuda")
        Z.embed_lookup(e, ids, w, out)
        return float((out.double() * act.double()).sum())

    h = 0.5
    for r, c in [(0, 0), (1, 5), (4, 2), (2, 3)]:
        up, down = table.clone(), table.clone()
        up[r, c] += h
        down[r, c] -= h
        d = (f(up) - f(down)) / (2 * h)
        # both sums of at most 9 * 6 products of size <= 3 * 5 * 5, rounded
        # to fp32 once per product
        assert abs(d - float(grad[r, c])) <= 2 * tokens * dim * 75 * U / h


def test_smallgrid_build_matches():
    """The build that splits every call over several launches."""
    ids = make_ids("zipf", 3000, 5000, 18)
    act, table = values((3000, 200), BF16, 19), values((5000, 200), BF16, 20)
    e = Z.make_embed(3000, 5000, 200, scale=2.0)
    ws = torch.empty(Z.zs_embed_workspace_bytes(e), dtype=torch.uint8, device="cuda")
    res = []
    for path in (Z.LIB_PATH, Z.SMALLGRID_LIB_PATH):
        with Z.library(path):
            out = torch.empty((3000, 200), dtype=BF16, device="cuda")
            grad = torch.empty((5000, 200), dtype=BF16, device="cuda")
            Z.embed_lookup(e, ids, table, out)
            Z.embed_grad(e, ids, act, grad, ws)
            Z.embed_grad(e, ids, act, grad, ws, accumulate=True)
            res.append((out, grad))
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])


def test_binding_refusals():
    e = Z.make_embed(4, 10, 8)
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    table = torch.zeros((10, 8), dtype=BF16, device="cuda")
    out = torch.zeros((4, 8), dtype=BF16, device="cuda")
    ws = torch.empty(Z.zs_embed_workspace_bytes(e), dtype=torch.uint8, device="cuda")
    for bad in (dict(ids=ids.int()), dict(ids=ids[:3]), dict(table=table.float()),
                dict(table=table[:9]), dict(out=out[:, :7]), dict(out=out.cpu()),
                dict(out=torch.zeros((8, 4), dtype=BF16, device="cuda").t())):
        kw = dict(ids=ids, table=table, out=out) | bad
        with pytest.raises(ValueError):
            Z.embed_lookup(e, kw["ids"], kw["table"], kw["out"])
    with pytest.raises(Z.ZSError) as err:
        Z.embed_grad(e, ids, out, table, ws[:-16])
    assert err.value.code == Z.ZS_EWORKSPACE
