"""MI355X sharded optimizer step (ZeRO-1/2/3, FSDP) -- Python binding.

Argument marshalling only: every function forwards to the C ABI of
``libzero_shard.so`` (declared in ``include/zero_shard.h``) with the same
name.  PyTorch tensors serve as device memory and streams; all arithmetic
runs in the library's HIP kernels.  There is no fallback: if the library is
missing, importing the entry points raises.
"""
from __future__ import annotations

import contextlib
import ctypes as C
import math
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libzero_shard.so")
# test build: at most 65,536 threads per launch (every entry point splits early)
# and the step's streaming loads at every size
SMALLGRID_LIB_PATH = os.path.join(_HERE, "libzero_shard_smallgrid.so")

ZS_OK = 0
ZS_EINVAL_PSI = -1
ZS_EINVAL_ND = -2
ZS_EINVAL_RANK = -3
ZS_EINVAL_LAYOUT = -4
ZS_EALIGN = -5
ZS_EINVAL_HPARAM = -6
ZS_EINVAL_STAGE = -7
ZS_ENULL = -8
ZS_EUNSUPPORTED = -9
ZS_EWORKSPACE = -10
ZS_ELAUNCH = -11
ZS_EINVAL_REDUCE = -12
ZS_EZERO_TOKENS = -13
ZS_EINVAL_UNITS = -14
ZS_ESCRATCH = -15
ZS_EINVAL_EMBED = -16
ZS_EINVAL_DISTILL = -17
ZS_EINVAL_TENSORS = -18
ZS_EINVAL_RELPOS = -19
ZS_SCRATCH_BYTES = 16 << 20
ZS_GRAD_BF16 = 0
ZS_GRAD_F32 = 1
ZS_MAX_RANKS = 64
ZS_OUT_GATHER = 0
ZS_OUT_SHARD = 1
ZS_BF16 = 0
ZS_F32 = 1
ZS_ID_I32 = 0
ZS_ID_I64 = 1
ZS_EMBED_MAX = 1 << 24
ZS_DISTILL_MAX_K = 1024
ZS_TENSORS_MAX = 1 << 24
ZS_RELPOS_MAX_BUCKETS = 256
ZS_RELPOS_FAR = 1 << 29


class ZSError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {zs_strerror(code)} (code {code})")
        self.code = code


class zs_shard(C.Structure):
    _fields_ = [("psi", C.c_int64), ("n_d", C.c_int32), ("rank", C.c_int32),
                ("align", C.c_int64), ("shard_len", C.c_int64), ("shard_offset", C.c_int64),
                ("valid_len", C.c_int64), ("stage", C.c_int32), ("out_mode", C.c_int32)]

    def __repr__(self):
        return ("zs_shard(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_)
                + ")")


class zs_adamw(C.Structure):
    _fields_ = [("lr", C.c_double), ("beta1", C.c_double), ("beta2", C.c_double),
                ("eps", C.c_double), ("weight_decay", C.c_double), ("step", C.c_int64),
                ("max_grad_norm", C.c_double)]


class zs_reduce(C.Structure):
    _fields_ = [("grad_dtype", C.c_int32), ("micro", C.c_int32), ("micro_count", C.c_int32),
                ("reserved", C.c_int32), ("rank_tokens", C.POINTER(C.c_int64))]


class zs_embed(C.Structure):
    _fields_ = [("tokens", C.c_int64), ("rows", C.c_int64), ("first_row", C.c_int64),
                ("dim", C.c_int64), ("table_pitch", C.c_int64), ("act_pitch", C.c_int64),
                ("id_dtype", C.c_int32), ("table_dtype", C.c_int32), ("act_dtype", C.c_int32),
                ("reserved", C.c_int32), ("scale", C.c_double)]


class zs_distill(C.Structure):
    _fields_ = [("rows", C.c_int64), ("vocab", C.c_int64), ("logits_pitch", C.c_int64),
                ("grad_pitch", C.c_int64), ("k", C.c_int32), ("logits_dtype", C.c_int32),
                ("teacher_dtype", C.c_int32), ("id_dtype", C.c_int32),
                ("temperature", C.c_double), ("alpha", C.c_double), ("scale", C.c_double)]


class zs_targets(C.Structure):
    _fields_ = [("teacher_ids", C.c_void_p), ("teacher_logits", C.c_void_p),
                ("teacher_lse", C.c_void_p), ("labels", C.c_void_p)]


class zs_tensor(C.Structure):
    _fields_ = [("in_", C.c_void_p), ("out", C.c_void_p), ("rows", C.c_int64),
                ("cols", C.c_int64), ("in_pitch", C.c_int64), ("out_pitch", C.c_int64),
                ("in_dtype", C.c_int32), ("out_dtype", C.c_int32)]


class zs_tensors(C.Structure):
    _fields_ = [("count", C.c_int64), ("elements", C.c_int64), ("bytes", C.c_int64),
                ("chunks", C.c_int64), ("chunk_bytes", C.c_int64), ("plan_bytes", C.c_int64),
                ("has_out", C.c_int32), ("stamp", C.c_uint32)]


class zs_relpos(C.Structure):
    _fields_ = [("batch", C.c_int64), ("heads", C.c_int64), ("queries", C.c_int64),
                ("keys", C.c_int64), ("in_pitch", C.c_int64 * 3), ("out_pitch", C.c_int64 * 3),
                ("table_pitch", C.c_int64), ("query_start", C.c_int64),
                ("max_distance", C.c_int64), ("buckets", C.c_int32),
                ("bidirectional", C.c_int32), ("causal", C.c_int32), ("dtype", C.c_int32),
                ("table_dtype", C.c_int32), ("id_dtype", C.c_int32), ("scale", C.c_double)]


_lib = None


def _open(path: str):
    """Load one build of the library and declare its entry points."""
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with __graft_entry__.build(); "
                          "there is no CPU fallback")
    L = C.CDLL(path)
    P, vp, i32, i64, f64 = C.POINTER, C.c_void_p, C.c_int32, C.c_int64, C.c_double
    L.zs_layout.argtypes = [i64, i32, i32, i64, i32, i32, P(zs_shard)]
    L.zs_layout.restype = C.c_int
    L.zs_workspace_bytes.argtypes = [P(zs_shard)]
    L.zs_workspace_bytes.restype = C.c_size_t
    L.zs_state_bytes.argtypes = [f64, i32, i32, f64]
    L.zs_state_bytes.restype = f64
    L.zs_comm_bytes.argtypes = [f64, i32, i32, f64]
    L.zs_comm_bytes.restype = f64
    L.shard_grad_sqnorm.argtypes = [P(zs_shard), vp, vp, vp, C.c_size_t, vp, i32, vp]
    L.shard_grad_sqnorm.restype = C.c_int
    L.zs_workspace_bytes_units.argtypes = [P(zs_shard), i32]
    L.zs_workspace_bytes_units.restype = C.c_size_t
    L.shard_grad_sqnorm_units.argtypes = [P(zs_shard), i32, vp, vp, vp, C.c_size_t, vp,
                                          i32, vp]
    L.shard_grad_sqnorm_units.restype = C.c_int
    L.shard_grad_reduce.argtypes = [P(zs_shard), P(zs_reduce), vp, vp, vp, C.c_size_t,
                                    vp, i32, vp]
    L.shard_grad_reduce.restype = C.c_int
    L.zero_shard_step.argtypes = [P(zs_shard), P(zs_adamw), vp, vp, vp, f64, vp, vp, vp,
                                  vp, vp]
    L.zero_shard_step.restype = C.c_int
    L.shard_pack_gather.argtypes = [P(zs_shard), vp, vp, vp]
    L.shard_pack_gather.restype = C.c_int
    L.zs_strerror.argtypes = [C.c_int]
    L.zs_strerror.restype = C.c_char_p
    L.shard_grad_sqnorm_noalloc.argtypes = [P(zs_shard), vp, vp, vp, i32, vp]
    L.shard_grad_sqnorm_noalloc.restype = C.c_int
    L.embed_lookup.argtypes = [P(zs_embed), vp, vp, vp, vp]
    L.embed_lookup.restype = C.c_int
    L.zs_embed_workspace_bytes.argtypes = [P(zs_embed)]
    L.zs_embed_workspace_bytes.restype = C.c_size_t
    L.embed_grad.argtypes = [P(zs_embed), vp, vp, vp, i32, vp, C.c_size_t, vp]
    L.embed_grad.restype = C.c_int
    L.zs_distill_workspace_bytes.argtypes = [P(zs_distill)]
    L.zs_distill_workspace_bytes.restype = C.c_size_t
    L.distill_loss.argtypes = [P(zs_distill), vp, P(zs_targets), vp, vp, vp, vp, i32, vp,
                               C.c_size_t, vp]
    L.distill_loss.restype = C.c_int
    L.distill_grad.argtypes = [P(zs_distill), vp, P(zs_targets), vp, vp, vp, vp]
    L.distill_grad.restype = C.c_int
    L.distill_loss_grad.argtypes = [P(zs_distill), vp, P(zs_targets), vp, vp, vp, vp, vp, vp,
                                    i32, vp, C.c_size_t, vp]
    L.distill_loss_grad.restype = C.c_int
    L.zs_tensors_layout.argtypes = [vp, i64, P(zs_tensors)]
    L.zs_tensors_layout.restype = C.c_int
    L.zs_tensors_plan.argtypes = [vp, P(zs_tensors), vp, C.c_size_t]
    L.zs_tensors_plan.restype = C.c_int
    L.tensors_sqnorm.argtypes = [P(zs_tensors), vp, vp, vp, i32, vp]
    L.tensors_sqnorm.restype = C.c_int
    L.tensors_clip.argtypes = [P(zs_tensors), vp, f64, vp, f64, vp]
    L.tensors_clip.restype = C.c_int
    L.tensors_clip_norm.argtypes = [P(zs_tensors), vp, f64, vp, vp, i32, vp]
    L.tensors_clip_norm.restype = C.c_int
    L.relpos_bias.argtypes = [P(zs_relpos), vp, vp, vp, vp, vp, vp]
    L.relpos_bias.restype = C.c_int
    L.zs_relpos_workspace_bytes.argtypes = [P(zs_relpos)]
    L.zs_relpos_workspace_bytes.restype = C.c_size_t
    L.relpos_bias_grad.argtypes = [P(zs_relpos), vp, vp, vp, vp, vp, i32, vp, C.c_size_t, vp]
    L.relpos_bias_grad.restype = C.c_int
    L.zs_init.argtypes = []
    L.zs_init.restype = C.c_int
    return L


def lib():
    """Load libzero_shard.so; raise if it has not been built."""
    global _lib
    if _lib is None:
        _lib = _open(LIB_PATH)
    return _lib


@contextlib.contextmanager
def library(path: str):
    """Route every call of this module through another build of the same
    ABI (the small-grid test build) while the context is open."""
    global _lib
    saved = lib()
    _lib = _open(path)
    try:
        yield _lib
    finally:
        _lib = saved


def zs_strerror(code: int) -> str:
    return lib().zs_strerror(code).decode()


def _check(rc: int, what: str) -> None:
    if rc != ZS_OK:
        raise ZSError(rc, what)


_F32 = ("float32",)
_F64 = ("float64",)
_I64 = ("int64",)
_B16 = ("int16", "bfloat16", "uint16")      # bf16 bit patterns
_ANY = None
_dtype_names = {}       # torch dtype -> its name


def _dtype_name(dtype) -> str:
    name = _dtype_names.get(dtype)
    if name is None:
        name = _dtype_names[dtype] = str(dtype).replace("torch.", "")
    return name


def _ptr(t, what: str = "buffer", dtypes=_ANY, min_numel: int = 0):
    """Device address of a tensor, an int address, or None.

    A torch tensor must have one of `dtypes` (torch dtype names; None: any),
    be contiguous, hold at least `min_numel` elements (what the call reads or
    writes through it) and live on the GPU; otherwise ValueError, before the
    C ABI is called.  An int is passed through unchecked."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not hasattr(t, "data_ptr"):
        raise TypeError(f"{what}: a torch tensor, an int device address or None is required")
    if dtypes is not None and _dtype_name(t.dtype) not in dtypes:
        raise ValueError(f"{what}: dtype {_dtype_name(t.dtype)}, expected "
                         f"{' or '.join(dtypes)}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: the tensor must be contiguous")
    if t.numel() < min_numel:
        raise ValueError(f"{what}: {t.numel()} elements, the call needs {min_numel}")
    if not t.is_cuda:
        raise ValueError(f"{what}: a GPU tensor is required (got {t.device})")
    return t.data_ptr()


def _bytes_ptr(t, what: str, nbytes: int):
    """As _ptr for a buffer of any dtype that must hold `nbytes` bytes."""
    if t is not None and not isinstance(t, int) and hasattr(t, "numel"):
        if t.numel() * t.element_size() < nbytes:
            raise ValueError(f"{what}: {t.numel() * t.element_size()} bytes, the call needs "
                             f"{nbytes}")
    return _ptr(t, what)


def _out_len(s: "zs_shard") -> int:
    """Elements of param_out the step or the pack writes up to: the slot
    [shard_offset, shard_offset + shard_len) of the gather buffer, or the
    rank's own shard."""
    return s.shard_len + (s.shard_offset if s.out_mode == ZS_OUT_GATHER else 0)


_torch = None


def _cuda():
    """torch.cuda, imported by the first call that needs it."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch.cuda


def _current_stream(device) -> int:
    # the same handle without building a Stream object (2.7 us a call)
    raw = getattr(_torch._C, "_cuda_getCurrentRawStream", None)
    return raw(device) if raw is not None else _torch.cuda.current_stream().cuda_stream


def _stream(stream):
    if stream is None:
        cuda = _cuda()
        if cuda.is_initialized():
            return _current_stream(cuda.current_device())
        return cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _slices(grad_slices, count: int, valid_len: int = 0, dtypes=_B16):
    """The host array of device pointers the C ABI reads `count` entries of
    (each slice tensor must hold valid_len elements of `dtypes`)."""
    if grad_slices is None:
        return None
    if len(grad_slices) != count:
        raise ValueError(f"{len(grad_slices)} gradient slice pointers given, {count} needed")
    arr = (C.c_void_p * count)(*[_ptr(g, f"grad_slices[{i}]", dtypes, valid_len)
                                 for i, g in enumerate(grad_slices)])
    return arr


# ---- host calls ------------------------------------------------------------------

def zs_init() -> None:
    """Per-device set-up of the current device (before capturing library
    calls into a HIP graph)."""
    _check(lib().zs_init(), "zs_init")


def zs_layout(psi: int, n_d: int, rank: int, align: int, stage: int = 2,
              out_mode: int = ZS_OUT_GATHER) -> zs_shard:
    s = zs_shard()
    _check(lib().zs_layout(psi, n_d, rank, align, stage, out_mode, C.byref(s)), "zs_layout")
    return s


def zs_workspace_bytes(s: zs_shard) -> int:
    return lib().zs_workspace_bytes(C.byref(s))


def zs_state_bytes(psi, n_d, stage, K=12.0) -> float:
    return lib().zs_state_bytes(float(psi), n_d, stage, float(K))


def zs_comm_bytes(psi, n_d, stage, bytes_per_elem=2.0) -> float:
    return lib().zs_comm_bytes(float(psi), n_d, stage, float(bytes_per_elem))


def adamw(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=1,
          max_grad_norm=0.0) -> zs_adamw:
    return zs_adamw(lr, beta1, beta2, eps, weight_decay, int(step), max_grad_norm)


# ---- device calls (enqueue on `stream`; torch tensors or raw addresses) ------------

def shard_grad_sqnorm(s: zs_shard, grad_slices, mean_out, workspace, sqnorm_out,
                      accumulate: bool = False, stream=None, workspace_bytes=None) -> None:
    if workspace_bytes is None:
        workspace_bytes = (workspace.numel() * workspace.element_size()
                           if hasattr(workspace, "numel") else zs_workspace_bytes(s))
    V = s.valid_len
    _check(lib().shard_grad_sqnorm(C.byref(s), _slices(grad_slices, s.n_d, V),
                                   _ptr(mean_out, "mean_out", _F32, V),
                                   _bytes_ptr(workspace, "workspace", workspace_bytes),
                                   workspace_bytes, _ptr(sqnorm_out, "sqnorm_out", _F64, 1),
                                   1 if accumulate else 0, _stream(stream)),
           "shard_grad_sqnorm")


def shard_grad_sqnorm_noalloc(s: zs_shard, grad_slices, mean_out, sqnorm_out,
                              accumulate: bool = False, stream=None) -> None:
    """shard_grad_sqnorm without a workspace argument: the library's static
    per-device scratch array holds the block partials (no allocation)."""
    V = s.valid_len
    _check(lib().shard_grad_sqnorm_noalloc(C.byref(s), _slices(grad_slices, s.n_d, V),
                                           _ptr(mean_out, "mean_out", _F32, V),
                                           _ptr(sqnorm_out, "sqnorm_out", _F64, 1),
                                           1 if accumulate else 0, _stream(stream)),
           "shard_grad_sqnorm_noalloc")


def zs_workspace_bytes_units(s: zs_shard, units: int) -> int:
    return lib().zs_workspace_bytes_units(C.byref(s), units)


def shard_grad_sqnorm_units(s: zs_shard, grad_slices, mean_out, workspace, sqnorm_out,
                            accumulate: bool = False, stream=None, workspace_bytes=None) -> None:
    """grad_slices: flat list of units * n_d device pointers (unit-major);
    mean_out: None or a list of `units` fp32 buffers (entries may be None)."""
    units = len(grad_slices) // s.n_d
    if units * s.n_d != len(grad_slices):
        raise ValueError("grad_slices must hold units * n_d pointers")
    means = None
    if mean_out is not None:
        if len(mean_out) != units:
            raise ValueError("one mean buffer per unit")
        means = (C.c_void_p * units)(*[_ptr(m, f"mean_out[{u}]", _F32, s.valid_len)
                                       for u, m in enumerate(mean_out)])
    if workspace_bytes is None:
        workspace_bytes = (workspace.numel() * workspace.element_size()
                           if hasattr(workspace, "numel") else zs_workspace_bytes_units(s, units))
    _check(lib().shard_grad_sqnorm_units(C.byref(s), units,
                                         _slices(grad_slices, units * s.n_d, s.valid_len),
                                         means, _bytes_ptr(workspace, "workspace",
                                                           workspace_bytes),
                                         workspace_bytes, _ptr(sqnorm_out, "sqnorm_out", _F64, 1),
                                         1 if accumulate else 0, _stream(stream)),
           "shard_grad_sqnorm_units")


def make_reduce(grad_dtype: int = ZS_GRAD_BF16, micro: int = 0, micro_count: int = 1,
                rank_tokens=None):
    """A zs_reduce; the token array it points to is kept alive on it."""
    r = zs_reduce(grad_dtype, micro, micro_count, 0, None)
    if rank_tokens is not None:
        arr = (C.c_int64 * len(rank_tokens))(*[int(t) for t in rank_tokens])
        r.rank_tokens = C.cast(arr, C.POINTER(C.c_int64))
        r._tokens = arr
    return r


def shard_grad_reduce(s: zs_shard, r: zs_reduce, grad_slices, grad_out, workspace=None,
                      sqnorm_out=None, accumulate: bool = False, stream=None,
                      workspace_bytes=None) -> None:
    if workspace_bytes is None:
        workspace_bytes = (workspace.numel() * workspace.element_size()
                           if hasattr(workspace, "numel") else
                           (zs_workspace_bytes(s) if workspace is not None else 0))
    tokens = getattr(r, "_tokens", None)
    if r.rank_tokens and (tokens is None or len(tokens) != s.n_d):
        raise ValueError(f"rank_tokens must hold n_d = {s.n_d} counts")
    V = s.valid_len
    gtypes = _F32 if r.grad_dtype == ZS_GRAD_F32 else _B16
    _check(lib().shard_grad_reduce(C.byref(s), C.byref(r), _slices(grad_slices, s.n_d, V, gtypes),
                                   _ptr(grad_out, "grad_out", _F32, V),
                                   _bytes_ptr(workspace, "workspace", workspace_bytes),
                                   workspace_bytes, _ptr(sqnorm_out, "sqnorm_out", _F64, 1),
                                   1 if accumulate else 0, _stream(stream)),
           "shard_grad_reduce")


def zero_shard_step(s: zs_shard, h: zs_adamw, grad_slices=None, mean_in=None, sqnorm=None,
                    other_sqnorm: float = 0.0, master=None, exp_avg=None, exp_avg_sq=None,
                    param_out=None, stream=None) -> None:
    V = s.valid_len
    _check(lib().zero_shard_step(C.byref(s), C.byref(h), _slices(grad_slices, s.n_d, V),
                                 _ptr(mean_in, "mean_in", _F32, V),
                                 _ptr(sqnorm, "sqnorm", _F64, 1), float(other_sqnorm),
                                 _ptr(master, "master", _F32, V),
                                 _ptr(exp_avg, "exp_avg", _F32, V),
                                 _ptr(exp_avg_sq, "exp_avg_sq", _F32, V),
                                 _ptr(param_out, "param_out", _B16, _out_len(s)),
                                 _stream(stream)), "zero_shard_step")


def shard_pack_gather(s: zs_shard, master, param_out, stream=None) -> None:
    _check(lib().shard_pack_gather(C.byref(s), _ptr(master, "master", _F32, s.valid_len),
                                   _ptr(param_out, "param_out", _B16, _out_len(s)),
                                   _stream(stream)), "shard_pack_gather")


# ---- the vocabulary table: embedding lookup and gradient, distillation ----------------

_IDS = {ZS_ID_I32: ("int32",), ZS_ID_I64: ("int64",)}
_ELEM = {ZS_BF16: _B16, ZS_F32: _F32}


def _rows_fit(shape, rows: int, width: int, pitch: int) -> bool:
    """Whether the sizes of a contiguous tensor agree with `rows` rows of
    `width` elements, `pitch` apart.  Rows are one dimension or the last few
    ([T, heads, head_dim]); one dimension, sizes of 1 aside, is a flat buffer;
    several rows may lie in one dimension if the rows fill the tensor."""
    sizes = [n for n in shape if n != 1]
    if len(sizes) < 2 or rows < 1:
        return True
    total = math.prod(sizes)
    n = 1
    for size in reversed(sizes):
        n *= size
        if n == pitch or (n % pitch == 0 and n < total == rows * pitch):
            return True
        if rows == 1 and (n == width or width < n < total):
            return True
    return False


def _rows_ptr(t, what: str, dtypes, rows: int, width: int, pitch: int):
    """As _ptr for `rows` rows of `width` elements, `pitch` apart: either a
    contiguous tensor that holds them, or a 2-D view with that row stride.
    A tensor whose own rows are of another pitch is refused."""
    shape = getattr(t, "shape", ())
    if len(shape) > 1 and (shape[-1] != pitch or rows < 2):
        if len(shape) == 2 and not t.is_contiguous():
            if shape[0] < rows or shape[1] < width or (width > 1 and t.stride(1) != 1) \
                    or (rows > 1 and t.stride(0) != pitch):
                raise ValueError(f"{what}: shape {tuple(shape)} with strides {t.stride()}, the "
                                 f"call needs {rows} rows of {width} elements, {pitch} apart")
            # the checks of _ptr on its first row; the rows' extent is checked above
            return _ptr(t[0, :width], what, dtypes)
        if pitch > 0 and shape[-1] != pitch and not _rows_fit(shape, rows, width, pitch):
            raise ValueError(f"{what}: shape {tuple(shape)}, the call needs {rows} rows of "
                             f"{width} elements, {pitch} apart")
    return _ptr(t, what, dtypes, (rows - 1) * pitch + width if rows > 0 else 0)


def _stream_on(stream, *tensors):
    """The stream's handle.  The library works on the current device: tensors
    and streams of another one are refused (raw addresses and handles are not
    looked at)."""
    cuda = _cuda()
    if not cuda.is_initialized():
        return _stream(stream)          # no GPU tensor yet: _ptr refuses the others
    device = cuda.current_device()
    for t in tensors:
        if t is not None and not isinstance(t, int) and t.get_device() != device:
            raise ValueError(f"a tensor on GPU {t.get_device()}: the current device is {device}")
    if stream is None:
        return _current_stream(device)
    if getattr(stream, "device_index", device) != device:
        raise ValueError(f"a stream of GPU {stream.device_index}: the current device is {device}")
    return _stream(stream)


def _sized(workspace, workspace_bytes, size, desc):
    """(address, bytes) of a workspace argument; an address without bytes is
    taken to hold size(desc), what the call needs."""
    if workspace_bytes is None:
        workspace_bytes = (workspace.numel() * workspace.element_size()
                           if hasattr(workspace, "numel") else size(desc))
    return _bytes_ptr(workspace, "workspace", workspace_bytes), workspace_bytes


def make_embed(tokens: int, rows: int, dim: int, first_row: int = 0, table_pitch=None,
               act_pitch=None, id_dtype: int = ZS_ID_I64, table_dtype: int = ZS_BF16,
               act_dtype: int = ZS_BF16, scale: float = 1.0) -> zs_embed:
    return zs_embed(tokens, rows, first_row, dim, dim if table_pitch is None else table_pitch,
                    dim if act_pitch is None else act_pitch, id_dtype, table_dtype, act_dtype, 0,
                    float(scale))


def zs_embed_workspace_bytes(e: zs_embed) -> int:
    return lib().zs_embed_workspace_bytes(C.byref(e))


def embed_lookup(e: zs_embed, ids, table, out, stream=None) -> None:
    _check(lib().embed_lookup(
        C.byref(e), _ptr(ids, "ids", _IDS.get(e.id_dtype), e.tokens),
        _rows_ptr(table, "table", _ELEM.get(e.table_dtype), e.rows, e.dim, e.table_pitch),
        _rows_ptr(out, "out", _ELEM.get(e.act_dtype), e.tokens, e.dim, e.act_pitch),
        _stream_on(stream, ids, table, out)), "embed_lookup")


def embed_grad(e: zs_embed, ids, grad_out, grad_table, workspace, accumulate: bool = False,
               stream=None, workspace_bytes=None) -> None:
    """The gradient of embed_lookup: grad_out are the T gradients of its rows,
    grad_table (of e.table_dtype) receives the table's."""
    ws, nbytes = _sized(workspace, workspace_bytes, zs_embed_workspace_bytes, e)
    _check(lib().embed_grad(
        C.byref(e), _ptr(ids, "ids", _IDS.get(e.id_dtype), e.tokens),
        _rows_ptr(grad_out, "grad_out", _ELEM.get(e.act_dtype), e.tokens, e.dim, e.act_pitch),
        _rows_ptr(grad_table, "grad_table", _ELEM.get(e.table_dtype), e.rows, e.dim,
                  e.table_pitch),
        1 if accumulate else 0, ws, nbytes,
        _stream_on(stream, ids, grad_out, grad_table, workspace)), "embed_grad")


def make_distill(rows: int, vocab: int, k: int, logits_pitch=None, grad_pitch=None,
                 logits_dtype: int = ZS_BF16, teacher_dtype: int = ZS_F32,
                 id_dtype: int = ZS_ID_I64, temperature: float = 1.0, alpha: float = 1.0,
                 scale: float = 1.0) -> zs_distill:
    return zs_distill(rows, vocab, vocab if logits_pitch is None else logits_pitch,
                      vocab if grad_pitch is None else grad_pitch, k, logits_dtype, teacher_dtype,
                      id_dtype, float(temperature), float(alpha), float(scale))


def zs_distill_workspace_bytes(d: zs_distill) -> int:
    return lib().zs_distill_workspace_bytes(C.byref(d))


def _targets(d: zs_distill, teacher_ids, teacher_logits, teacher_lse, labels) -> zs_targets:
    ids, rows, k = _IDS.get(d.id_dtype), d.rows, d.k
    return zs_targets(
        _rows_ptr(teacher_ids, "teacher_ids", ids, rows, k, k),
        _rows_ptr(teacher_logits, "teacher_logits", _ELEM.get(d.teacher_dtype), rows, k, k),
        _ptr(teacher_lse, "teacher_lse", _F32, rows), _ptr(labels, "labels", ids, rows))


def _lse_ptr(d: zs_distill, t):
    return _rows_ptr(t, "lse", _F32, d.rows, 2, 2)


def _logits_ptr(d: zs_distill, t, what: str, pitch: int):
    return _rows_ptr(t, what, _ELEM.get(d.logits_dtype), d.rows, d.vocab, pitch)


def distill_loss(d: zs_distill, logits, teacher_ids, teacher_logits, loss, lse, teacher_lse=None,
                 labels=None, loss_sum=None, counted=None, accumulate: bool = False,
                 workspace=None, stream=None, workspace_bytes=None) -> None:
    """Row losses (loss: fp32[T], lse: fp32[T, 2]); loss_sum: one fp32 and
    counted: one int64, or None."""
    t = _targets(d, teacher_ids, teacher_logits, teacher_lse, labels)
    ws, nbytes = _sized(workspace, workspace_bytes, zs_distill_workspace_bytes, d)
    _check(lib().distill_loss(
        C.byref(d), _logits_ptr(d, logits, "logits", d.logits_pitch), C.byref(t),
        _ptr(loss, "loss", _F32, d.rows), _lse_ptr(d, lse),
        _ptr(loss_sum, "loss_sum", _F32, 1), _ptr(counted, "counted", _I64, 1),
        1 if accumulate else 0, ws, nbytes,
        _stream_on(stream, logits, teacher_ids, teacher_logits, teacher_lse, labels, loss, lse,
                   loss_sum, counted, workspace)), "distill_loss")


def distill_grad(d: zs_distill, logits, teacher_ids, teacher_logits, lse, grad, teacher_lse=None,
                 labels=None, row_grad=None, stream=None) -> None:
    """The logits' gradient from the lse of distill_loss; grad may be logits."""
    t = _targets(d, teacher_ids, teacher_logits, teacher_lse, labels)
    _check(lib().distill_grad(
        C.byref(d), _logits_ptr(d, logits, "logits", d.logits_pitch), C.byref(t),
        _lse_ptr(d, lse), _ptr(row_grad, "row_grad", _F32, d.rows),
        _logits_ptr(d, grad, "grad", d.grad_pitch),
        _stream_on(stream, logits, teacher_ids, teacher_logits, teacher_lse, labels, lse, row_grad,
                   grad)), "distill_grad")


def distill_loss_grad(d: zs_distill, logits, teacher_ids, teacher_logits, loss, grad,
                      teacher_lse=None, labels=None, lse=None, row_grad=None, loss_sum=None,
                      counted=None, accumulate: bool = False, workspace=None, stream=None,
                      workspace_bytes=None) -> None:
    """distill_loss and distill_grad in one call; grad may be logits."""
    t = _targets(d, teacher_ids, teacher_logits, teacher_lse, labels)
    ws, nbytes = _sized(workspace, workspace_bytes, zs_distill_workspace_bytes, d)
    _check(lib().distill_loss_grad(
        C.byref(d), _logits_ptr(d, logits, "logits", d.logits_pitch), C.byref(t),
        _ptr(loss, "loss", _F32, d.rows), _lse_ptr(d, lse),
        _ptr(row_grad, "row_grad", _F32, d.rows),
        _logits_ptr(d, grad, "grad", d.grad_pitch), _ptr(loss_sum, "loss_sum", _F32, 1),
        _ptr(counted, "counted", _I64, 1), 1 if accumulate else 0, ws, nbytes,
        _stream_on(stream, logits, teacher_ids, teacher_logits, teacher_lse, labels, loss, lse,
                   row_grad, grad, loss_sum, counted, workspace)), "distill_loss_grad")


# ---- the position-bias table: bias by buckets, and its gradient ------------------------

def make_relpos(heads: int, queries: int, keys: int, buckets: int = 32, max_distance: int = 128,
                batch: int = 1, bidirectional: bool = True, causal: bool = False,
                query_start: int = 0, scale: float = 1.0, dtype: int = ZS_BF16,
                table_dtype: int = ZS_F32, id_dtype: int = ZS_ID_I64, in_pitch=None,
                out_pitch=None, table_pitch=None) -> zs_relpos:
    """in_pitch, out_pitch: elements from one sequence, head, query to the next
    ([batch, heads, queries, keys] without gaps if not given)."""
    plain = (heads * queries * keys, queries * keys, keys)
    triple = C.c_int64 * 3
    return zs_relpos(batch, heads, queries, keys, triple(*(in_pitch or plain)),
                     triple(*(out_pitch or plain)),
                     heads if table_pitch is None else table_pitch, query_start, max_distance,
                     buckets, 1 if bidirectional else 0, 1 if causal else 0, dtype, table_dtype,
                     id_dtype, float(scale))


def zs_relpos_workspace_bytes(r: zs_relpos) -> int:
    return lib().zs_relpos_workspace_bytes(C.byref(r))


def _places_ptr(r: zs_relpos, t, what: str, pitch):
    """Address of a [batch, heads, queries, keys] tensor with these pitches (a
    batch of one may be left out), or of a flat buffer that holds them."""
    if t is None or isinstance(t, int):
        return t
    sizes = (r.batch, r.heads, r.queries, r.keys)
    if getattr(t, "shape", None) == sizes and t.stride() == (*pitch, 1):
        # the usual tensor: what _ptr checks beside its extent
        if t.is_cuda and _dtype_name(t.dtype) in _ELEM.get(r.dtype, ()):
            return t.data_ptr()
    need = 0
    if min(sizes) > 0:
        need = r.keys + sum((n - 1) * p for n, p in zip(sizes, pitch))
    shape, strides = getattr(t, "shape", ()), ()
    if len(shape) == 4 or (len(shape) == 3 and r.batch == 1):
        strides = t.stride()
        if len(shape) == 3:
            shape, strides = (1, *shape), (0, *strides)
        if tuple(shape) != sizes or need and any(
                n > 1 and s != p for n, s, p in zip(sizes, strides, (*pitch, 1))):
            raise ValueError(f"{what}: shape {tuple(t.shape)} with strides {t.stride()}, the call "
                             f"needs {sizes} with strides {(*pitch, 1)}")
        if need == 0 or t.is_contiguous():
            return _ptr(t, what, _ELEM.get(r.dtype))
        # the checks of _ptr on its first place; the extent is the shape's
        return _ptr(t[(slice(0, 1),) * t.dim()], what, _ELEM.get(r.dtype))
    if len(shape) != 1:
        raise ValueError(f"{what}: shape {tuple(shape)}, the call needs {sizes}")
    return _ptr(t, what, _ELEM.get(r.dtype), need)


def _relpos_table(r: zs_relpos, t, what: str):
    return _rows_ptr(t, what, _ELEM.get(r.table_dtype), r.buckets, r.heads, r.table_pitch)


def relpos_bias(r: zs_relpos, table, out, scores=None, key_lengths=None, query_starts=None,
                stream=None) -> None:
    """The bias of every place of [batch, heads, queries, keys] into out, added to
    scale * scores where they are given (out may be scores); -Inf where a key is
    not seen.  table: [buckets, heads]."""
    ids = _IDS.get(r.id_dtype)
    _check(lib().relpos_bias(
        C.byref(r), _relpos_table(r, table, "table"),
        _places_ptr(r, scores, "scores", r.in_pitch),
        _ptr(key_lengths, "key_lengths", ids, r.batch),
        _ptr(query_starts, "query_starts", ids, r.batch),
        _places_ptr(r, out, "out", r.out_pitch),
        _stream_on(stream, table, scores, key_lengths, query_starts, out)), "relpos_bias")


def relpos_bias_grad(r: zs_relpos, grad, grad_table, workspace, grad_scores=None,
                     key_lengths=None, query_starts=None, accumulate: bool = False, stream=None,
                     workspace_bytes=None) -> None:
    """The gradient of relpos_bias: grad is that of its output, grad_table (of
    r.table_dtype) receives the table's, grad_scores (may be grad) the scores'."""
    ws, nbytes = _sized(workspace, workspace_bytes, zs_relpos_workspace_bytes, r)
    ids = _IDS.get(r.id_dtype)
    _check(lib().relpos_bias_grad(
        C.byref(r), _places_ptr(r, grad, "grad", r.in_pitch),
        _ptr(key_lengths, "key_lengths", ids, r.batch),
        _ptr(query_starts, "query_starts", ids, r.batch),
        _relpos_table(r, grad_table, "grad_table"),
        _places_ptr(r, grad_scores, "grad_scores", r.out_pitch), 1 if accumulate else 0, ws,
        nbytes, _stream_on(stream, grad, key_lengths, query_starts, grad_table, grad_scores,
                           workspace)), "relpos_bias_grad")


# ---- many tensors: the global norm and the clip ---------------------------------------

_TENSOR_TYPES = {"bfloat16": ZS_BF16, "float32": ZS_F32}


def _rows_of(t):
    """(rows, cols, pitch) of a tensor whose elements fill memory in any order of
    its dimensions, or whose rows (the dimensions but the one of stride 1 or
    those that are contiguous with it) are evenly apart; None for any other."""
    dims = sorted(((st, n) for st, n in zip(t.stride(), t.shape) if n != 1))
    if t.numel() == 0:
        return 0, 0, 0
    cols = 1
    while dims and dims[0][0] == cols:
        cols *= dims.pop(0)[1]
    if not dims:
        return 1, cols, cols
    pitch, rows = dims[0][0], 1
    for st, n in dims:
        if st != pitch * rows:
            return None
        rows *= n
    return (rows, cols, pitch) if pitch >= cols else None


class Tensors:
    """A list of tensors as tensors_sqnorm, tensors_clip and tensors_clip_norm
    take it: the struct, its plan on the GPU, and the tensors themselves, whose
    memory the plan names.  Make a new one where a tensor is replaced by another
    (a gradient that was set to None and made anew), or keep gradients where they
    are: a list of 1500 takes 2 to 3 ms to make.  One call at a time uses a
    list (its plan holds their partial sums), and the list lives until its calls
    have ended on the GPU."""

    def __init__(self, struct, plan, tensors, out, device):
        self.struct, self.plan, self.tensors, self.out = struct, plan, tensors, out
        self.device = device
        self.refs = C.byref(struct), plan.data_ptr()      # what every call hands over


def _tensor_entry(i, t, o):
    for what, x in (("tensors", t), ("out", o)):
        if not hasattr(x, "data_ptr"):
            raise TypeError(f"{what}[{i}]: a torch tensor is required")
        if _dtype_name(x.dtype) not in _TENSOR_TYPES:
            raise ValueError(f"{what}[{i}]: dtype {_dtype_name(x.dtype)}, expected bfloat16 or "
                             "float32")
        if not x.is_cuda:
            raise ValueError(f"{what}[{i}]: a GPU tensor is required (got {x.device})")
    rows = _rows_of(t)
    if rows is None:
        raise ValueError(f"tensors[{i}]: shape {tuple(t.shape)} with strides {t.stride()} is not "
                         "rows of contiguous elements evenly apart")
    other = rows
    if o is not t:
        if o.shape != t.shape:
            raise ValueError(f"out[{i}]: shape {tuple(o.shape)}, the tensor's is {tuple(t.shape)}")
        other = _rows_of(o)
        if other is None or not _same_order(t, o) or (
                other[:2] != rows[:2] and 1 not in (other[0], rows[0])):
            raise ValueError(f"out[{i}]: strides {o.stride()}, the tensor's are {t.stride()}: not "
                             "the same rows of elements in the same order")
        # one without gaps is cut into the other's rows
        if rows[0] < other[0]:
            rows = (other[0], other[1], other[1])
        elif other[0] < rows[0]:
            other = (rows[0], rows[1], rows[1])
    return zs_tensor(t.data_ptr(), o.data_ptr(), rows[0], rows[1], rows[2], other[2],
                     _TENSOR_TYPES[_dtype_name(t.dtype)], _TENSOR_TYPES[_dtype_name(o.dtype)])


def _same_order(t, o) -> bool:
    """Whether the dimensions larger than 1 have their strides in the same order."""
    dims = [d for d, n in enumerate(t.shape) if n != 1]
    return (sorted(dims, key=lambda d: t.stride(d)) == sorted(dims, key=lambda d: o.stride(d)))


def make_tensors(tensors, out=None) -> Tensors:
    """The list of GPU tensors (bfloat16 or float32, of any sizes) whose global
    norm is taken; out: where each goes when it is clipped, a list of tensors of
    the same shapes (views of a flat buffer, say), or None: in place.

    A tensor's elements may be in any order in memory as long as they fill it
    (a transposed gradient), or its rows may be evenly apart.  None may be written
    where another is read or written (the same tensor twice, in place)."""
    tensors = list(tensors)
    out = tensors if out is None else list(out)
    if len(out) != len(tensors):
        raise ValueError(f"{len(tensors)} tensors, {len(out)} out")
    cuda = _cuda()
    kinds = {_torch.bfloat16: ZS_BF16, _torch.float32: ZS_F32}
    # zs_tensor's seven words a tensor
    words, devices = [], set()
    for i, (t, o) in enumerate(zip(tensors, out)):
        kind, other = kinds.get(getattr(t, "dtype", None)), kinds.get(getattr(o, "dtype", None))
        if (kind is not None and other is not None and t.is_cuda and o.is_cuda
                and t.is_contiguous() and o.is_contiguous() and t.shape == o.shape):
            n = t.numel()
            words += (t.data_ptr(), o.data_ptr(), 1, n, n, n, kind | other << 32)
        else:
            e = _tensor_entry(i, t, o)
            words += (e.in_ or 0, e.out or 0, e.rows, e.cols, e.in_pitch, e.out_pitch,
                      e.in_dtype | e.out_dtype << 32)
        devices.add(t.get_device())
        devices.add(o.get_device())
    device = cuda.current_device()
    for d in devices:
        if d != device:
            raise ValueError(f"a tensor on GPU {d}: the current device is {device}")
    arr = (C.c_int64 * max(len(words), 1))(*words)
    struct = zs_tensors()
    _check(lib().zs_tensors_layout(arr, len(tensors), C.byref(struct)), "zs_tensors_layout")
    host = _torch.empty(struct.plan_bytes, dtype=_torch.uint8)
    _check(lib().zs_tensors_plan(arr, C.byref(struct), host.data_ptr(), struct.plan_bytes),
           "zs_tensors_plan")
    # pageable memory: the copy has ended when .to returns
    return Tensors(struct, host.to(f"cuda:{device}"), tensors, out, device)


def _tensors_on(t: Tensors, stream, *scalars):
    return (*t.refs, _stream_on(stream, t.plan, *scalars))


def tensors_sqnorm(t: Tensors, sqnorm_out, tensor_sqnorms=None, accumulate: bool = False,
                   stream=None) -> None:
    """The squared norm of the whole list into sqnorm_out (one float64);
    tensor_sqnorms: float64[count] for each tensor's own, or None."""
    struct, plan, stream = _tensors_on(t, stream, sqnorm_out, tensor_sqnorms)
    _check(lib().tensors_sqnorm(
        struct, plan, _ptr(sqnorm_out, "sqnorm_out", _F64, 1),
        _ptr(tensor_sqnorms, "tensor_sqnorms", _F64, t.struct.count),
        1 if accumulate else 0, stream), "tensors_sqnorm")


def tensors_clip(t: Tensors, max_norm: float, sqnorm, other_sqnorm: float = 0.0,
                 stream=None) -> None:
    """Every tensor times the coefficient of the global squared norm *sqnorm +
    other_sqnorm, as zero_shard_step takes it."""
    struct, plan, stream = _tensors_on(t, stream, sqnorm)
    _check(lib().tensors_clip(struct, plan, float(max_norm), _ptr(sqnorm, "sqnorm", _F64, 1),
                              float(other_sqnorm), stream), "tensors_clip")


def tensors_clip_norm(t: Tensors, max_norm: float, sqnorm_out, tensor_sqnorms=None,
                      accumulate: bool = False, stream=None) -> None:
    """tensors_sqnorm, then tensors_clip by what it left in sqnorm_out."""
    struct, plan, stream = _tensors_on(t, stream, sqnorm_out, tensor_sqnorms)
    _check(lib().tensors_clip_norm(
        struct, plan, float(max_norm), _ptr(sqnorm_out, "sqnorm_out", _F64, 1),
        _ptr(tensor_sqnorms, "tensor_sqnorms", _F64, t.struct.count),
        1 if accumulate else 0, stream), "tensors_clip_norm")


def build(verbose: bool = False) -> str:
    from . import _build
    return _build.build(verbose)
