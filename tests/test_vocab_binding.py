"""The binding's own checks of the vocabulary-table calls, on the CPU: what a
tensor's shape says about its rows is held against the call's row widths and
pitches.  A CPU tensor whose shape is accepted is refused last, for not being
on the GPU, so every case ends before the C ABI."""
import pytest
import torch

import fsdp_sharded_optimizer_zero_amd as Z

BF16 = torch.bfloat16
ACCEPTED = "GPU tensor is required"
REFUSED = "apart"


def rows_ptr(shape, rows, width, pitch, dtype=BF16):
    return Z._rows_ptr(torch.zeros(shape, dtype=dtype), "rows", None, rows, width, pitch)


# shape of a contiguous tensor, rows, width, pitch
HOLDS = [((6, 50), 6, 50, 50), ((6, 56), 6, 50, 56),
         ((8, 50), 6, 50, 50),                              # more rows than asked
         ((300,), 6, 50, 50), ((5 * 56 + 50,), 6, 50, 56),  # a flat buffer
         ((1, 300), 6, 50, 50), ((300, 1), 6, 50, 50),      # the same, by its sizes
         ((2, 3, 50), 6, 50, 50), ((6, 5, 10), 6, 50, 50), ((2, 3, 5, 10), 6, 50, 50),
         ((1, 6, 56), 6, 50, 56), ((1, 56), 1, 50, 50), ((4, 56), 1, 50, 50),
         ((5, 10), 1, 50, 50),
         ((3, 100), 6, 50, 50), ((2, 150), 6, 50, 50),      # [batch, length x 50]
         ((6, 1), 6, 1, 1), ((0, 50), 0, 50, 50), ((4, 56), 0, 50, 50)]
# the padded rows of a contiguous tensor at the pitch of narrower ones, and others
WRONG = [((6, 56), 6, 50, 50), ((50, 6), 6, 50, 50), ((2, 3, 56), 6, 50, 50),
         ((6, 100), 6, 50, 50), ((12, 25), 6, 50, 56), ((2, 300), 6, 50, 50), ((5, 8), 1, 20, 20)]


@pytest.mark.parametrize("shape,rows,width,pitch", HOLDS)
def test_rows_of_the_calls_pitch_are_accepted(shape, rows, width, pitch):
    with pytest.raises(ValueError, match=ACCEPTED):
        rows_ptr(shape, rows, width, pitch)


@pytest.mark.parametrize("shape,rows,width,pitch", WRONG)
def test_rows_of_another_pitch_are_refused(shape, rows, width, pitch):
    with pytest.raises(ValueError, match=REFUSED):
        rows_ptr(shape, rows, width, pitch)


@pytest.mark.parametrize("rows,pitch,ok", [(6, 56, True), (6, 50, False), (6, 64, False),
                                           (1, 50, True), (1, 56, True), (0, 50, True)])
def test_views_of_padded_rows(rows, pitch, ok):
    """The first 50 of 56 columns: rows 56 apart, or one row."""
    view = torch.zeros((6, 56), dtype=BF16)[:, :50]
    with pytest.raises(ValueError, match=ACCEPTED if ok else "apart|contiguous"):
        Z._rows_ptr(view, "rows", None, rows, 50, pitch)


def test_padded_tables_and_logits_need_their_pitch():
    """Each tensor of rows of each call: 8 columns wider than the default
    pitch is refused, with the pitch named it is accepted."""
    T, R, D, K = 5, 30, 16, 2
    table = torch.zeros((R, D + 8), dtype=BF16)
    act, ok = torch.zeros((T, D + 8), dtype=BF16), torch.zeros((T, D), dtype=BF16)

    def calls(**pitch):
        e = Z.make_embed(T, R, D, **{k: v for k, v in pitch.items() if k[0] in "ta"})
        d = Z.make_distill(T, R, K, **{k: v for k, v in pitch.items() if k[0] in "lg"})
        w = dict(table=(e.rows, e.dim, e.table_pitch), act=(e.tokens, e.dim, e.act_pitch),
                 logits=(d.rows, d.vocab, d.logits_pitch), grad=(d.rows, d.vocab, d.grad_pitch))
        return lambda name, t: Z._rows_ptr(t, name, None, *w[name])

    plain, padded = calls(), calls(table_pitch=D + 8, act_pitch=D + 8, logits_pitch=R + 8,
                                   grad_pitch=R + 8)
    wide = torch.zeros((T, R + 8), dtype=BF16)
    for name, t in (("table", table), ("act", act), ("logits", wide), ("grad", wide)):
        with pytest.raises(ValueError, match=REFUSED):
            plain(name, t)
        with pytest.raises(ValueError, match=ACCEPTED):
            padded(name, t)
    # as the entry points are called: the first tensor of rows is what is wrong
    e, d = Z.make_embed(T, R, D), Z.make_distill(T, R, K)
    at = 4096           # an address, not looked at
    for call in (lambda: Z.embed_lookup(e, at, table, ok),
                 lambda: Z.embed_grad(e, at, act, table, 0),
                 lambda: Z.distill_loss(d, wide, at, at, 0, 0, workspace=0),
                 lambda: Z.distill_grad(d, wide, at, at, 0, wide),
                 lambda: Z.distill_loss_grad(d, wide, at, at, 0, wide, workspace=0)):
        with pytest.raises(ValueError, match=REFUSED):
            call()


class OnGpu:
    """A CPU tensor that says it is on a GPU, for checks that stop before the
    library is called."""

    def __init__(self, t, device=0):
        self._t, self._device = t, device

    is_cuda = property(lambda self: True)

    def get_device(self):
        return self._device

    def __getattr__(self, name):
        return getattr(self._t, name)


def stopped(monkeypatch):
    """The library's calls raise: all checks of the binding were passed."""
    class Library:
        def __getattr__(self, name):
            def call(*args):
                raise ArithmeticError("called")
            return call

    sizes = {n: getattr(Z, n) for n in ("zs_embed_workspace_bytes", "zs_distill_workspace_bytes")}
    real = Z.lib()
    monkeypatch.setattr(Z, "lib", lambda: Library())
    for name in sizes:
        monkeypatch.setattr(Z, name, lambda s, f=getattr(real, name): f(Z.C.byref(s)))


def distill_tensors(T=6, V=40, K=4):
    f = torch.float32
    return Z.make_distill(T, V, K), dict(
        logits=torch.zeros((T, V), dtype=BF16), teacher_ids=torch.zeros((T, K), dtype=torch.int64),
        teacher_logits=torch.zeros((T, K), dtype=f), teacher_lse=torch.zeros(T, dtype=f),
        labels=torch.zeros(T, dtype=torch.int64), loss=torch.zeros(T, dtype=f),
        lse=torch.zeros((T, 2), dtype=f), grad=torch.zeros((T, V), dtype=BF16),
        loss_sum=torch.zeros(1, dtype=f), counted=torch.zeros(1, dtype=torch.int64),
        workspace=torch.zeros(1 << 16, dtype=torch.uint8))


def distill_calls(d, x):
    """The three calls on the same tensors."""
    t = dict(teacher_lse=x["teacher_lse"], labels=x["labels"])
    sums = dict(loss_sum=x["loss_sum"], counted=x["counted"], workspace=x["workspace"])
    who = (x["logits"], x["teacher_ids"], x["teacher_logits"])
    return {"loss": lambda: Z.distill_loss(d, *who, x["loss"], x["lse"], **t, **sums, stream=0),
            "grad": lambda: Z.distill_grad(d, *who, x["lse"], x["grad"], **t, stream=0),
            "both": lambda: Z.distill_loss_grad(d, *who, x["loss"], x["grad"], lse=x["lse"], **t,
                                                **sums, stream=0)}


def on_gpu(x, **device):
    return {k: OnGpu(t, device.get(k, 0)) for k, t in x.items()}


@pytest.mark.parametrize("name,shape", [
    ("teacher_ids", (6, 5)), ("teacher_logits", (6, 5)), ("teacher_ids", (3, 2, 8)),
    ("teacher_logits", (6, 8)), ("teacher_ids", (4, 7)), ("lse", (6, 3)), ("lse", (3, 5))])
def test_teacher_entries_of_another_count_are_refused(monkeypatch, name, shape):
    """[T, k'] tensors at k entries a row, and an lse that is not [T, 2]."""
    stopped(monkeypatch)
    d, x = distill_tensors()
    x[name] = torch.zeros(shape, dtype=x[name].dtype)
    for call in distill_calls(d, on_gpu(x)).values():
        with pytest.raises(ValueError, match=REFUSED):
            call()


@pytest.mark.parametrize("shape", [(6, 4), (2, 3, 4), (24,), (8, 4), (1, 24), (2, 12)])
def test_teacher_entries_of_the_calls_count_are_accepted(monkeypatch, shape):
    stopped(monkeypatch)
    d, x = distill_tensors()
    for name in ("teacher_ids", "teacher_logits"):
        x[name] = torch.zeros(shape, dtype=x[name].dtype)
    x["lse"] = torch.zeros((12,))
    for call in distill_calls(d, on_gpu(x)).values():
        with pytest.raises(ArithmeticError):
            call()


def current(monkeypatch, device):
    class Cuda:
        is_initialized = staticmethod(lambda: True)
        current_device = staticmethod(lambda: device)

    monkeypatch.setattr(Z, "_cuda", lambda: Cuda)


@pytest.mark.parametrize("call", ["loss", "grad", "both"])
def test_every_tensor_of_another_device_is_refused(monkeypatch, call):
    """One tensor after the other on GPU 1 while GPU 0 is current."""
    stopped(monkeypatch)
    current(monkeypatch, 0)
    d, x = distill_tensors()
    with pytest.raises(ArithmeticError):
        distill_calls(d, on_gpu(x))[call]()
    unused = {"loss": {"grad"}, "grad": {"loss", "loss_sum", "counted", "workspace"}, "both": set()}
    for name in set(x) - unused[call]:
        with pytest.raises(ValueError, match="current device"):
            distill_calls(d, on_gpu(x, **{name: 1}))[call]()


def test_a_stream_of_another_device_is_refused(monkeypatch):
    """The kernels of a call are those of the current device."""
    class Stream:
        cuda_stream = 77

        def __init__(self, device):
            self.device_index = device

    current(monkeypatch, 0)
    assert Z._stream_on(Stream(0)) == 77 and Z._stream_on(5) == 5
    with pytest.raises(ValueError, match="current device"):
        Z._stream_on(Stream(1))
