"""The norm and the clip of many tensors against 64-bit forms.

The squared norm is a sum of non-negative fp64 terms, each square exact: its
relative error is at most the longest chain of additions times 2^-53.  A thread
of a piece adds at most its share of the piece, a few hundred elements at these
sizes, then come the wave, the block, the list; 4096 additions bound them all.
The clip is exact: the coefficient is correctly rounded operations in double on
the device's own squared norm, the product one fp32 rounding, the output
another."""
import math

import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_zero_amd as Z

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
REL = 4096 * 2.0 ** -53
GUARD = 37


def scalar(value=0.0):
    return torch.full((1,), value, dtype=F64, device="cuda")


def sq_sum(t):
    return math.fsum((t.detach().cpu().double() ** 2).reshape(-1).tolist()) \
        if t.numel() < 200000 else float(t.double().square().sum())


def coef_of(q, max_norm, other=0.0):
    with np.errstate(all="ignore"):
        c = np.float64(max_norm) / (np.sqrt(np.float64(q) + np.float64(other)) + 1e-6)
    return np.float32(1.0 if c > 1.0 else c)


def clipped(t, coef, dtype):
    return (t.float() * float(coef)).to(dtype) if coef == coef else \
        torch.full_like(t, math.nan, dtype=dtype)


def same(a, b):
    return torch.equal(torch.nan_to_num(a.float(), nan=12345.0),
                       torch.nan_to_num(b.float(), nan=12345.0))


def make(sizes, types, seed=0, std=1e-2, skew=0):
    """Tensors with `skew` elements before each, so that they begin anywhere."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for k, n in enumerate(sizes):
        numel = math.prod(n) if isinstance(n, tuple) else n
        off = skew * (k + 1) % 8 if skew else 0
        buf = torch.randn(numel + off, generator=g, device="cuda") * (std * (1 + k % 3))
        t = buf.to(types[k % len(types)])[off:off + numel]
        out.append(t.view(n) if isinstance(n, tuple) else t)
    return out


def flat_views(tensors, dtype, gap=0):
    """Views of a guarded flat buffer, `gap` elements apart."""
    total = sum(t.numel() + gap for t in tensors)
    buf = torch.full((total + GUARD,), -7.0, dtype=dtype, device="cuda")
    views, at = [], gap
    mask = torch.ones_like(buf, dtype=torch.bool)
    for t in tensors:
        views.append(buf[at:at + t.numel()].view(t.shape))
        mask[at:at + t.numel()] = False
        at += t.numel() + gap
    return buf, views, mask


def check(tensors, out=None, max_norm=0.5, prior=None, other=0.0, mask=None, buf=None):
    src = [t.clone() for t in tensors]
    T = Z.make_tensors(tensors, out)
    q, each = scalar(prior or 0.0), torch.full((max(len(tensors), 1),), -1.0, dtype=F64,
                                               device="cuda")
    Z.tensors_sqnorm(T, q, each, accumulate=prior is not None)
    torch.cuda.synchronize()
    want = [sq_sum(t) for t in src]
    total = math.fsum(want) + (prior or 0.0)
    got = float(q)
    assert abs(got - total) <= REL * total, (got, total)
    for k, w in enumerate(want):
        assert abs(float(each[k]) - w) <= REL * w, (k, float(each[k]), w)
    for t, s in zip(tensors, src):
        assert torch.equal(t, s), "the norm writes no tensor"
    Z.tensors_clip(T, max_norm, q, other_sqnorm=other)
    torch.cuda.synchronize()
    coef = coef_of(got, max_norm, other)
    dst = tensors if out is None else out
    for k, (s, o) in enumerate(zip(src, dst)):
        assert torch.equal(o, clipped(s, coef, o.dtype)), k
    if mask is not None:
        assert bool((buf[mask] == -7.0).all()), "written outside the tensors"
    return T, q, coef


SIZES = [[], [0], [1], [1, 0, 2, 3], [7, 8, 9, 15, 16, 17, 255, 256, 257], [2047, 2048, 2049],
         [4096, 16384, 16385, 1], [(33, 65), (5, 1), (1, 1), (3, 4, 5)], [100003, 50, 8, 0, 1],
         [3] * 300, [5, 700] * 400, [1 << 20] * 30, [(1 << 24) + 3, 1, (1 << 22) - 1]]


@pytest.mark.parametrize("sizes", SIZES, ids=range(len(SIZES)))
@pytest.mark.parametrize("types,out,skew", [((BF16,), F32, 0), ((F32,), F32, 1), ((BF16,), BF16, 3),
                                            ((F32, BF16), BF16, 1), ((BF16, F32), F32, 5)])
def test_lists(sizes, types, out, skew):
    tensors = make(sizes, types, seed=len(sizes), skew=skew)
    buf, views, mask = flat_views(tensors, out, gap=skew % 2)
    check(tensors, views, mask=mask, buf=buf)


@pytest.mark.parametrize("types", [(BF16,), (F32,), (BF16, F32)])
@pytest.mark.parametrize("prior,other", [(None, 0.0), (3.0, 0.0), (0.0, 2.5), (1e300, 1e300)])
def test_in_place_prior_and_other(types, prior, other):
    tensors = make([1000, (64, 65), 3, 40000], types, seed=5, skew=1)
    check(tensors, prior=prior, other=other)


def test_one_call_is_both():
    tensors = make([1000, 5, 70000], (BF16, F32), seed=6)
    outs = [torch.empty_like(t) for t in tensors]
    T, q, _ = check(tensors, outs)
    q2, each2 = scalar(), torch.empty(3, dtype=F64, device="cuda")
    outs2 = [torch.empty_like(t) for t in tensors]
    T2 = Z.make_tensors(tensors, outs2)
    Z.tensors_clip_norm(T2, 0.5, q2, each2)
    assert torch.equal(q, q2) and all(torch.equal(a, b) for a, b in zip(outs, outs2))
    q3 = q2.clone()
    Z.tensors_clip_norm(T2, 0.5, q3, accumulate=True)
    assert abs(float(q3) - 2 * float(q2)) <= REL * float(q3)
    coef = coef_of(float(q3), 0.5)
    assert all(torch.equal(o, clipped(t, coef, t.dtype)) for t, o in zip(tensors, outs2))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_within_the_limit_in_place_nothing_changes(dtype):
    """A coefficient of 1 leaves every bit, subnormals and -0 among them; out of
    place it copies."""
    tensors = make([5000, 3], (dtype,), seed=7)
    tensors[0][:4] = torch.tensor([-0.0, 1e-40, -1e-40, 0.0])
    bits = [t.clone() for t in tensors]
    view = torch.int16 if dtype == BF16 else torch.int32
    q = scalar()
    Z.tensors_clip_norm(Z.make_tensors(tensors), 1e6, q)
    assert all(torch.equal(a.view(view), b.view(view)) for a, b in zip(tensors, bits))
    outs = [torch.empty_like(t) for t in tensors]
    Z.tensors_clip_norm(Z.make_tensors(tensors, outs), 1e6, q)
    assert all(torch.equal(a.view(view), b.view(view)) for a, b in zip(outs, bits))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("where", [0, 1, 2])
def test_nan_and_inf_propagate(bad, where):
    tensors = make([300, 20000, 7], (F32, BF16), seed=8)
    tensors[where][-1] = bad
    src = [t.clone() for t in tensors]
    q, each = scalar(), torch.zeros(3, dtype=F64, device="cuda")
    Z.tensors_clip_norm(Z.make_tensors(tensors), 1.0, q, each)
    want = math.nan if math.isnan(bad) else math.inf
    assert str(float(q)) == str(want) and str(float(each[where])) == str(want)
    assert all(math.isfinite(float(each[k])) for k in range(3) if k != where)
    coef = math.nan if math.isnan(bad) else 0.0
    for s, t in zip(src, tensors):
        assert same(t, (s.float() * coef).to(t.dtype))


def test_small_and_large_values():
    """Squares that fp32 could not hold."""
    t = torch.tensor([1e-30, 3e-38, 1e-41, 0.0], device="cuda")
    big = torch.tensor([3e38, -3e38], device="cuda").to(BF16)
    check([t], max_norm=1e-31)
    check([t, big, t.clone()], max_norm=1.0)


LAYOUTS = [lambda d: torch.randn((40, 90), device="cuda").to(d)[:, :77],
           lambda d: torch.randn((40, 90), device="cuda").to(d)[3:, 5:6],
           lambda d: torch.randn((50, 60), device="cuda").to(d).t(),
           lambda d: torch.randn((3, 50, 60), device="cuda").to(d)[:, 7:20],
           lambda d: torch.randn((2, 30000), device="cuda").to(d)[:, 1:25001],
           lambda d: torch.randn((5000, 3), device="cuda").to(d)[:, :2],
           lambda d: torch.randn((6, 8, 10), device="cuda").to(d).permute(2, 0, 1),
           lambda d: torch.randn((700, 2050), device="cuda").to(d)[:, 1:2050]]


@pytest.mark.parametrize("k", range(len(LAYOUTS)))
@pytest.mark.parametrize("dtype,out", [(BF16, F32), (F32, BF16), (BF16, BF16), (F32, F32)])
def test_strides(k, dtype, out):
    """Rows apart, transposed gradients: clipped in place, and into dense or
    padded tensors; what lies between the rows stays."""
    torch.manual_seed(k)
    t = LAYOUTS[k](dtype)
    base = t._base if t._base is not None else t
    around = base.clone()
    check([t, torch.ones(3, device="cuda")])
    mine = torch.zeros_like(base, dtype=torch.bool)
    mine.as_strided(t.shape, t.stride(), t.storage_offset()).fill_(True)
    assert torch.equal(base[~mine], around[~mine]), "in place: written between the rows"
    like = torch.empty_strided(t.shape, t.stride(), dtype=out, device="cuda")
    check([t], [like])
    if t.stride() == tuple(sorted(t.stride(), reverse=True)):
        check([t], [torch.empty(t.shape, dtype=out, device="cuda")])
        wide = torch.full((*t.shape[:-1], t.shape[-1] + 3), -7.0, dtype=out, device="cuda")
        if t.dim() == 2:
            check([t], [wide[:, :-3]])
            assert bool((wide[:, -3:] == -7.0).all())
            dense = t.contiguous()
            check([dense], [wide[:, :-3]])


@pytest.mark.parametrize("sizes", [[100, 5000], [100003] * 5, [3] * 300])
def test_same_bits_every_time(sizes):
    """The order of the sums is fixed, whichever block ends last, and the plan
    is left as it was found."""
    tensors = make(sizes, (BF16, F32), seed=9)
    T = Z.make_tensors(tensors)
    plan = T.plan.clone()
    first = None
    for _ in range(20):
        q, each = scalar(), torch.empty(len(sizes), dtype=F64, device="cuda")
        Z.tensors_sqnorm(T, q, each)
        now = (q.clone(), each.clone())
        first = first or now
        assert torch.equal(now[0], first[0]) and torch.equal(now[1], first[1])
    assert torch.equal(T.plan[:256], plan[:256])


def test_small_grid_build():
    """Launches of at most 256 blocks: a list of more pieces takes several."""
    tensors = make([1 << 20] * 9 + [5, 0], (BF16, F32), seed=10)
    with Z.library(Z.SMALLGRID_LIB_PATH):
        T, _, _ = check(tensors, [torch.empty_like(t) for t in tensors])
        assert T.struct.chunks > 2 * 256


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_more_than_32_bits_of_elements(dtype):
    """One tensor past 2^31 elements, between small ones; in place."""
    n = (1 << 31) + 12345
    t = torch.zeros(n, dtype=dtype, device="cuda")
    for at in (0, (1 << 31) - 1, 1 << 31, n - 1):
        t[at] = 3.0
    small = [torch.full((5,), 2.0, device="cuda"), torch.full((3,), 1.0, device="cuda")]
    T = Z.make_tensors([small[0], t, small[1]])
    q, each = scalar(), torch.empty(3, dtype=F64, device="cuda")
    Z.tensors_clip_norm(T, 1.0, q, each)
    assert float(q) == 20.0 + 36.0 + 3.0 and each.tolist() == [20.0, 36.0, 3.0]
    coef = coef_of(59.0, 1.0)
    value = clipped(torch.tensor([3.0], device="cuda"), coef, dtype)
    for at in (0, (1 << 31) - 1, 1 << 31, n - 1):
        assert float(t[at]) == float(value[0])
    assert int(torch.count_nonzero(t)) == 4
    assert torch.equal(small[1], clipped(torch.ones(3, device="cuda"), coef, F32))


def test_many_tensors():
    """More tensors than pieces a list of large ones is cut into."""
    check(make([1 + 37 * i % 90 for i in range(9001)], (BF16, F32), seed=11))


def test_captured_and_replayed():
    """A graph of norm, clip and both, replayed with new gradients and eager
    work between; the first call of the process's list may be captured."""
    Z.zs_init()
    tensors = make([1000, 70, 30000, 1 << 21], (BF16, F32), seed=12)
    flat, views, _ = flat_views(tensors, F32)
    T = Z.make_tensors(tensors, views)
    place = [t.clone() for t in tensors]
    P = Z.make_tensors(place)
    q, q2 = scalar(), scalar()
    each = torch.zeros(4, dtype=F64, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Z.tensors_sqnorm(T, q, each)
        Z.tensors_clip(T, 0.3, q)
        Z.tensors_clip_norm(P, 0.2, q2)
    for k in range(5):
        fresh = make([1000, 70, 30000, 1 << 21], (BF16, F32), seed=20 + k)
        for t, p, f in zip(tensors, place, fresh):
            t.copy_(f)
            p.copy_(f)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = math.fsum(sq_sum(f) for f in fresh)
        assert abs(float(q) - want) <= REL * want and abs(float(q2) - want) <= REL * want
        coef, coef2 = coef_of(float(q), 0.3), coef_of(float(q2), 0.2)
        for f, v, p in zip(fresh, views, place):
            assert torch.equal(v, clipped(f, coef, F32))
            assert torch.equal(p, clipped(f, coef2, p.dtype))
        eager = scalar()
        Z.tensors_sqnorm(T, eager)
        assert torch.equal(eager, q)


def test_lists_on_two_streams():
    """Two lists at once, each on its own stream: a plan is its call's own."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets = [make([40000, 9, 1 << 20], (BF16,), seed=30 + k) for k in range(2)]
    outs = [[torch.empty_like(t, dtype=F32) for t in s] for s in sets]
    lists = [Z.make_tensors(s, o) for s, o in zip(sets, outs)]
    qs = [scalar() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(30):
        for st, T, q in zip(streams, lists, qs):
            Z.tensors_clip_norm(T, 0.1, q, stream=st)
    torch.cuda.synchronize()
    for s, o, q in zip(sets, outs, qs):
        coef = coef_of(float(q), 0.1)
        assert all(torch.equal(x, clipped(t, coef, F32)) for t, x in zip(s, o))


def test_norm_adds_to_a_shards():
    """A shard's pass and a list into one scalar: the step and the clip read it."""
    s = Z.zs_layout(100003, 4, 1, 8, 2)
    rows = (torch.randn((4, s.shard_len), device="cuda") * 1e-2).to(BF16)
    ws = torch.empty(Z.zs_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    q = scalar()
    Z.shard_grad_sqnorm(s, [rows[r] for r in range(4)], None, ws, q)
    shard = float(q)
    tensors = make([771, 50], (F32,), seed=13)
    Z.tensors_sqnorm(Z.make_tensors(tensors), q, accumulate=True)
    want = shard + math.fsum(sq_sum(t) for t in tensors)
    assert abs(float(q) - want) <= REL * want


def test_binding_refuses():
    tensors = make([10, 20], (F32,))
    T = Z.make_tensors(tensors)
    with pytest.raises(ValueError, match="sqnorm_out"):
        Z.tensors_sqnorm(T, torch.zeros(1, device="cuda"))
    with pytest.raises(ValueError, match="tensor_sqnorms"):
        Z.tensors_sqnorm(T, scalar(), torch.zeros(1, dtype=F64, device="cuda"))
    with pytest.raises(ValueError, match="GPU -1|GPU tensor"):
        Z.tensors_clip(T, 1.0, torch.zeros(1, dtype=F64))
    with pytest.raises(Z.ZSError, match="hyperparameter"):
        Z.tensors_clip(T, 0.0, scalar())
    with pytest.raises(ValueError, match="shape"):
        Z.make_tensors(tensors, [tensors[0], tensors[0]])
    with pytest.raises(ValueError, match="float64"):
        Z.make_tensors([scalar()])


def test_columns_of_one_matrix_and_the_same_tensor_twice():
    """Three column slices of one gradient are three tensors; the same memory
    twice is refused."""
    fused = torch.randn((50, 96), device="cuda").to(BF16)
    parts = list(fused.split(32, dim=1))
    check(parts)
    with pytest.raises(Z.ZSError, match="zs_tensor"):
        Z.make_tensors([parts[0], fused])
    with pytest.raises(Z.ZSError, match="zs_tensor"):
        Z.make_tensors([parts[0], parts[0]])
    flat = torch.zeros(100, device="cuda")
    with pytest.raises(Z.ZSError, match="zs_tensor"):
        Z.make_tensors([parts[0][0], parts[1][0]], [flat[:32], flat[31:63]])


def test_tensors_of_another_device_are_refused(monkeypatch):
    tensors = make([10, 20], (F32,))
    T, q = Z.make_tensors(tensors), scalar()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in (lambda: Z.make_tensors(tensors), lambda: Z.tensors_sqnorm(T, q, stream=0),
                 lambda: Z.tensors_clip(T, 1.0, q, stream=0),
                 lambda: Z.tensors_clip_norm(T, 1.0, q, stream=0)):
        with pytest.raises(ValueError, match="current device"):
            call()


def test_a_list_outlives_the_callers_names():
    """The list keeps its tensors: what the caller lets go is not handed out anew."""
    T = Z.make_tensors(make([1 << 20, 5], (F32,), seed=14))
    want = math.fsum(sq_sum(t) for t in T.tensors)
    for _ in range(5):
        torch.full((1 << 20,), 7.0, device="cuda")
    q = scalar()
    Z.tensors_sqnorm(T, q)
    assert abs(float(q) - want) <= REL * want


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("max_norm", [1e150, 1.5e154, 1e300, 1.7976931348623157e308])
def test_an_infinite_norm_is_past_every_limit(dtype, max_norm):
    """In place, also with limits whose square is not finite: a list with an
    infinite element is clipped by 0, one without stays as it is."""
    fine = make([300, 20000, 7], (dtype,), seed=9)
    bits = [t.clone() for t in fine]
    q = scalar()
    Z.tensors_clip_norm(Z.make_tensors(fine), max_norm, q)
    assert all(torch.equal(a, b) for a, b in zip(fine, bits))
    # another rank's norm
    T = Z.make_tensors(fine)
    Z.tensors_clip(T, max_norm, q, other_sqnorm=math.inf)
    assert all(bool((t == 0).all()) for t in fine)
    tensors = make([300, 20000, 7], (dtype,), seed=9)
    tensors[1][-1] = math.inf
    outs = [torch.empty_like(t) for t in tensors]
    Z.tensors_clip_norm(Z.make_tensors(tensors, outs), max_norm, q)
    Z.tensors_clip_norm(Z.make_tensors(tensors), max_norm, q)
    assert float(q) == math.inf
    for k, (t, o) in enumerate(zip(tensors, outs)):
        assert same(t, o)
        assert bool((t.nan_to_num(nan=0.0) == 0).all())
        assert int(t.isnan().sum()) == (k == 1)
