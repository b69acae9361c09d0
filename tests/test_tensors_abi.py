"""Host-side checks of the calls on many tensors (no GPU needed): how a list is
cut into pieces, every documented argument error before anything is enqueued,
and what the binding reads from a tensor's strides.  Fake device addresses are
used, so the calls run only where no GPU is visible."""
import ctypes as C

import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_zero_amd as Z

no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="fake-address error paths run only without a GPU")
FAKE = 0x7F0000000000
SIZE = {Z.ZS_BF16: 2, Z.ZS_F32: 4}
PIECE = np.dtype([("in", "<u8"), ("out", "<u8"), ("in_pitch", "<i8"), ("out_pitch", "<i8"),
                  ("rows", "<i4"), ("cols", "<i4"), ("kind", "<i4"), ("tensor", "<i4")])


def entry(rows=1, cols=100, in_=FAKE, out=FAKE + (1 << 40), in_pitch=None, out_pitch=None,
          in_dtype=Z.ZS_BF16, out_dtype=Z.ZS_F32):
    return Z.zs_tensor(in_, out, rows, cols, cols if in_pitch is None else in_pitch,
                       cols if out_pitch is None else out_pitch, in_dtype, out_dtype)


def layout(entries, count=None):
    arr = (Z.zs_tensor * max(len(entries), 1))(*entries)
    t = Z.zs_tensors()
    rc = Z.lib().zs_tensors_layout(arr, len(entries) if count is None else count, C.byref(t))
    return rc, t, arr


def plan(entries):
    """The plan of the entries, moved apart in memory."""
    for i, e in enumerate(entries):
        place = e.in_ == e.out
        e.in_ = FAKE + (i << 37)
        e.out = e.in_ if place else (1 << 60) + (i << 37)
    rc, t, arr = layout(entries)
    assert rc == Z.ZS_OK
    host = np.full(t.plan_bytes, 0xAB, np.uint8)
    assert Z.lib().zs_tensors_plan(arr, C.byref(t), host.ctypes.data, host.nbytes) == Z.ZS_OK
    assert not host[:256].any(), "the counter starts at 0"
    pieces = host[256:256 + t.chunks * PIECE.itemsize].view(PIECE)
    first = 256 + -(-t.chunks * PIECE.itemsize // 256) * 256
    return t, pieces, host[first:first + 8 * (t.count + 1)].view(np.int64)


LISTS = [
    [],
    [entry(cols=0)],
    [entry(cols=1)],
    [entry(rows=0, cols=5), entry(cols=7), entry(cols=0), entry(cols=2049)],
    [entry(cols=c) for c in (2047, 2048, 2049, 16384, 16385, 65537)],
    [entry(rows=33, cols=65), entry(rows=33, cols=65, in_pitch=70), entry(rows=5, cols=1)],
    [entry(rows=7, cols=771, in_pitch=771, out_pitch=800, in_dtype=Z.ZS_F32)],
    [entry(rows=3, cols=50000, in_pitch=60000, out_pitch=50001)],
    [entry(rows=1000, cols=3, in_pitch=4, in_dtype=Z.ZS_F32, out_dtype=Z.ZS_BF16)],
    [entry(cols=100000, out=FAKE, out_dtype=Z.ZS_BF16), entry(cols=5000)],
    [entry(cols=1 << 31), entry(cols=(1 << 33) + 5, in_dtype=Z.ZS_F32)],
    [entry(rows=1 << 20, cols=1 << 12, in_pitch=1 << 13)],
    [entry(cols=1 + 37 * i % 500) for i in range(9000)],
]


@pytest.mark.parametrize("entries", LISTS, ids=range(len(LISTS)))
def test_pieces_cover_every_element_once(entries):
    t, pieces, first = plan(entries)
    assert t.count == len(entries) and t.chunks == len(pieces) == first[-1]
    assert t.elements == sum(e.rows * e.cols for e in entries) and t.has_out == (
        2 if all(e.in_ == e.out or e.rows * e.cols == 0 for e in entries) else 1)
    assert t.bytes == sum(e.rows * e.cols * SIZE[e.in_dtype] for e in entries)
    for i, e in enumerate(entries):
        mine = pieces[first[i]:first[i + 1]]
        assert (mine["tensor"] == i).all()
        isz, osz = SIZE[e.in_dtype], SIZE[e.out_dtype]
        assert (mine["kind"] == (e.in_dtype == Z.ZS_F32) + 2 * (e.out_dtype == Z.ZS_F32)
                + 4 * (e.in_ == e.out)).all()
        n = mine["rows"].astype(np.int64) * mine["cols"]
        assert n.sum() == e.rows * e.cols and (n > 0).all()
        wide = max(isz, osz) if e.out else isz
        assert (n * wide <= t.chunk_bytes * (2 if e.in_ == e.out else 1)).all()
        if e.rows * e.cols == 0:
            continue
        # pieces follow one another without a gap or an overlap, in both buffers
        off = (mine["in"] - np.uint64(e.in_)).astype(np.int64) // isz
        oof = (mine["out"] - np.uint64(e.out)).astype(np.int64) // osz
        dense = e.rows == 1 or (e.in_pitch == e.cols and e.out_pitch == e.cols)
        if dense:
            assert (mine["rows"] == 1).all()
            assert (off == np.concatenate([[0], np.cumsum(n)[:-1]])).all() and (oof == off).all()
            continue
        row, col = off // e.in_pitch, off % e.in_pitch
        assert (oof == row * e.out_pitch + col).all()
        many = mine["rows"] > 1
        assert (mine["in_pitch"][many] == e.in_pitch).all()
        assert (mine["out_pitch"][many] == e.out_pitch).all()
        assert (mine["cols"][many] == e.cols).all() and (col[many] == 0).all()
        place = row * e.cols + col
        assert (place == np.concatenate([[0], np.cumsum(n)[:-1]])).all()


BAD = [dict(rows=-1), dict(cols=-1), dict(in_dtype=2), dict(out_dtype=-1),
       dict(rows=2, in_pitch=99), dict(rows=2, out_pitch=99), dict(cols=1 << 61),
       dict(rows=1 << 31, cols=1 << 31), dict(rows=2, in_pitch=1 << 60),
       dict(out=FAKE, out_dtype=Z.ZS_F32),                          # in place, another type
       dict(out=FAKE, out_dtype=Z.ZS_BF16, rows=2, out_pitch=104)]  # in place, another pitch


@pytest.mark.parametrize("bad", BAD)
def test_entries_are_refused(bad):
    assert layout([entry(in_=FAKE + 4096, out=2 * FAKE), entry(**bad)])[0] == Z.ZS_EINVAL_TENSORS


def test_lists_are_refused():
    assert layout([entry(in_=None)])[0] == Z.ZS_ENULL
    assert layout([entry(in_=FAKE + 1)])[0] == Z.ZS_EALIGN
    assert layout([entry(out=FAKE + 2)])[0] == Z.ZS_EALIGN
    assert layout([entry()], count=-1)[0] == Z.ZS_EINVAL_TENSORS
    assert layout([entry()], count=Z.ZS_TENSORS_MAX + 1)[0] == Z.ZS_EUNSUPPORTED
    assert layout([entry(cols=1 << 59), entry(cols=1 << 59)])[0] == Z.ZS_EINVAL_TENSORS
    L = Z.lib()
    assert L.zs_tensors_layout(None, 1, C.byref(Z.zs_tensors())) == Z.ZS_ENULL
    assert L.zs_tensors_layout(None, 0, C.byref(Z.zs_tensors())) == Z.ZS_OK
    assert L.zs_tensors_layout(None, 0, None) == Z.ZS_ENULL
    # no element is read of a tensor without any
    assert layout([entry(cols=0, in_=None, out=None)])[0] == Z.ZS_OK
    rc, t, arr = layout([entry(), entry(in_=FAKE + 4096, out=None)])
    assert rc == Z.ZS_OK and t.has_out == 0
    host = np.zeros(t.plan_bytes, np.uint8)
    fill = lambda a, s, n=host.nbytes: L.zs_tensors_plan(a, C.byref(s), host.ctypes.data, n)
    assert fill(arr, t, host.nbytes - 1) == Z.ZS_EWORKSPACE
    other = layout([entry(), entry(in_=FAKE + 4096, cols=101, out=None)])
    assert fill(other[2], t) == Z.ZS_EINVAL_TENSORS       # another list's
    assert L.zs_tensors_plan(arr, C.byref(t), None, host.nbytes) == Z.ZS_ENULL
    assert L.zs_tensors_plan(arr, None, host.ctypes.data, host.nbytes) == Z.ZS_ENULL


def test_overlaps_are_refused():
    """An `out` that shares a byte with another tensor's `in` or `out`."""
    A = FAKE
    own = dict(in_dtype=Z.ZS_F32)
    place = lambda at, **kw: entry(in_=at, out=at, **own, **kw)
    go = lambda at, to, **kw: entry(in_=at, out=to, **own, **kw)
    B = A + (1 << 30)
    ok = [
        [place(A), place(A + 400)],
        [go(A, B), go(A, B + 400)],                                 # read twice
        [go(A, B), go(A + 200, B + 400)],
        [place(A, rows=5, cols=30, in_pitch=100, out_pitch=100),    # columns of a matrix
         place(A + 120, rows=5, cols=70, in_pitch=100, out_pitch=100)],
        [place(A + 120, rows=5, cols=70, in_pitch=100, out_pitch=100),
         place(A, rows=5, cols=30, in_pitch=100, out_pitch=100),
         place(A + 400 * 5, cols=100)],
        [place(A, rows=5, cols=30, in_pitch=100, out_pitch=100),    # one row beside them
         place(A + 400 * 2 + 120, cols=70)],
        [place(A, cols=0), place(A)],
    ]
    bad = [
        [place(A), place(A)],                                       # the same, twice
        [place(A), place(A + 396)],
        [go(A, B), go(A + 4000, B)],
        [go(A, A + 4)],                                             # onto itself, moved
        [go(A, B), go(B, B + 4000)],                                # reads what is written
        [go(B, B + 4000), go(A, B)],
        [place(A), go(A, B)],
        [place(A, rows=5, cols=30, in_pitch=100, out_pitch=100),
         place(A + 116, rows=5, cols=70, in_pitch=100, out_pitch=100)],
        [place(A, rows=5, cols=30, in_pitch=100, out_pitch=100),
         place(A + 120, rows=5, cols=71, in_pitch=100, out_pitch=100)],
        [place(A, rows=5, cols=30, in_pitch=100, out_pitch=100),
         place(A + 120, rows=5, cols=10, in_pitch=50, out_pitch=50)],
        [place(A, rows=5, cols=30, in_pitch=100, out_pitch=100), place(A + 1100, cols=100)],
        [place(A, cols=5000), place(A + 400, cols=1), place(A + 8000, cols=1)],
    ]
    for entries in ok:
        assert layout(entries)[0] == Z.ZS_OK, entries
    for entries in bad:
        assert layout(entries)[0] == Z.ZS_EINVAL_TENSORS, entries
        assert layout(entries[::-1])[0] == Z.ZS_EINVAL_TENSORS, entries


@no_gpu
def test_calls_are_refused():
    L = Z.lib()
    t = layout([entry()])[1]
    norms = layout([entry(out=None)])[1]

    def sq(t, plan=FAKE, out=FAKE, each=None):
        return L.tensors_sqnorm(None if t is None else C.byref(t), plan, out, each, 0, None)

    def clip(t, plan=FAKE, norm=1.0, q=FAKE, other=0.0):
        return L.tensors_clip(C.byref(t), plan, norm, q, other, None)

    def both(t, plan=FAKE, norm=1.0, out=FAKE, each=None):
        return L.tensors_clip_norm(C.byref(t), plan, norm, out, each, 0, None)

    assert sq(None) == Z.ZS_ENULL
    for call, name in ((sq, "out"), (clip, "q"), (both, "out")):
        assert call(t, plan=None) == Z.ZS_ENULL and call(t, plan=FAKE + 8) == Z.ZS_EALIGN
        assert call(t, **{name: None}) == Z.ZS_ENULL and call(t, **{name: FAKE + 4}) == Z.ZS_EALIGN
        for field, value in (("count", -1), ("chunks", 2), ("plan_bytes", 0), ("stamp", 1), ("has_out", 3),
                             ("count", Z.ZS_TENSORS_MAX + 1), ("elements", 0)):
            bad = Z.zs_tensors.from_buffer_copy(t)
            setattr(bad, field, value)
            assert call(bad) == Z.ZS_EINVAL_TENSORS, field
    assert sq(t, each=FAKE + 4) == Z.ZS_EALIGN and both(t, each=FAKE + 4) == Z.ZS_EALIGN
    for norm in (0.0, -1.0, float("nan"), float("inf")):
        assert clip(t, norm=norm) == Z.ZS_EINVAL_HPARAM and both(t, norm=norm) == Z.ZS_EINVAL_HPARAM
    assert clip(t, other=-1.0) == Z.ZS_EINVAL_HPARAM
    assert clip(norms) == Z.ZS_ENULL and both(norms) == Z.ZS_ENULL       # nothing to write to
    assert "zs_tensor" in Z.zs_strerror(Z.ZS_EINVAL_TENSORS)


@no_gpu
def test_nothing_to_clip_is_no_launch():
    empty = layout([entry(cols=0)])[1]
    assert Z.lib().tensors_clip(C.byref(empty), FAKE, 1.0, FAKE, 0.0, None) == Z.ZS_OK


# ---- the binding ------------------------------------------------------------------------

base = torch.zeros((6, 8, 10))
ROWS = [(base, (1, 480, 480)), (base.transpose(0, 2), (1, 480, 480)), (base[:, :, :7], (48, 7, 10)),
        (base[:, 2:5], (6, 30, 80)), (base[2], (1, 80, 80)), (base[:, 3], (6, 10, 80)),
        (base[:, :, 3], (48, 1, 10)), (base[:, :, :1], (48, 1, 10)), (base[:0], (0, 0, 0)),
        (base.permute(1, 2, 0), (1, 480, 480)), (base[1, 1, 1], (1, 1, 1)),
        (base[:, 2:5].transpose(0, 1), (6, 30, 80)),
        (base[::2, :, :], (3, 80, 160)), (base[:, :3, :7], None), (base[:, :, ::2], (240, 1, 2)),
        (torch.zeros(1).expand(5), None), (torch.zeros((4, 1)).expand(4, 5), None)]


@pytest.mark.parametrize("t,rows", ROWS, ids=range(len(ROWS)))
def test_rows_of_a_tensor(t, rows):
    assert Z._rows_of(t) == rows
    if rows and t.numel():
        # the rows name the tensor's elements, each once
        n, cols, pitch = rows
        flat = torch.arange(n)[:, None] * pitch + torch.arange(cols)
        own = t.storage_offset() + sum(
            torch.arange(k).reshape([-1 if i == d else 1 for i in range(t.dim())]) * s
            for d, (k, s) in enumerate(zip(t.shape, t.stride()))) if t.dim() else \
            torch.tensor([t.storage_offset()])
        assert torch.equal(flat.reshape(-1).sort().values + t.storage_offset(),
                           own.reshape(-1).sort().values)


def test_binding_refuses_lists():
    ok = torch.zeros(4)
    with pytest.raises(TypeError, match=r"tensors\[1\]"):
        Z.make_tensors([_Cuda(ok), 5])
    with pytest.raises(ValueError, match="float16"):
        Z.make_tensors([_Cuda(ok.half())])
    with pytest.raises(ValueError, match="GPU tensor"):
        Z.make_tensors([ok])
    with pytest.raises(ValueError, match="1 tensors, 2 out"):
        Z.make_tensors([ok], [ok, ok])
    wide = torch.zeros((4, 6))
    for t, o, what in ((torch.zeros(1).expand(5), None, "evenly apart"),
                       (ok, torch.zeros(5), "shape"),
                       (wide, torch.zeros((6, 4)).t(), "order"),
                       (wide[:, :4], torch.zeros((4, 4)).t(), "order"),
                       (torch.zeros((4, 3, 5))[:, :, :4], torch.zeros((4, 4, 4))[:, :3], "order")):
        with pytest.raises(ValueError, match=what):
            Z._tensor_entry(0, _Cuda(t), _Cuda(t) if o is None else _Cuda(o))
    # rows of one and none of the other's gaps
    e = Z._tensor_entry(0, _Cuda(wide[:, :4]), _Cuda(torch.zeros((4, 4))))
    assert (e.rows, e.cols, e.in_pitch, e.out_pitch) == (4, 4, 6, 4)
    e = Z._tensor_entry(0, _Cuda(torch.zeros((4, 4))), _Cuda(wide[:, :4]))
    assert (e.rows, e.cols, e.in_pitch, e.out_pitch) == (4, 4, 4, 6)
    e = Z._tensor_entry(0, _Cuda(torch.zeros((4, 6)).t()), _Cuda(torch.zeros((4, 6)).t()))
    assert (e.rows, e.cols) == (1, 24)


class _Cuda:
    """A CPU tensor that says it is on the GPU: the checks before the address."""

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return True if name == "is_cuda" else getattr(self.t, name)
