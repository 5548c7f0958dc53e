"""What the selector's binding hands to the C entries, in both of its forms: the Python one with host tensors
and the C calls recorded, the C one with stand-ins for tensors whose addresses are never read (every such call
is refused by the C entry on the host)."""
import importlib.machinery
import importlib.util

import pytest
import torch

INVALID = -1
BF, U8, I8, F32, I32, I64 = torch.bfloat16, torch.uint8, torch.int8, torch.float32, torch.int32, torch.int64


@pytest.fixture(scope="module")
def m():
    from mla_latent_cache_attention_gb300 import build
    build.build()
    import mla_latent_cache_attention_gb300 as mod
    mod.lib()
    return mod


class Declined:
    """A marshalling that serves nothing: every call takes its Python form."""
    insert = gather = scores = select = selected = staticmethod(lambda *a: None)


@pytest.fixture
def python_form(m, monkeypatch):
    """The Python form on host tensors: the C calls' names and arguments, instead of the calls."""
    calls = []
    monkeypatch.setattr(m, "_marshal", Declined())
    monkeypatch.setattr(m, "_cuda_device", lambda t: t.device)
    monkeypatch.setattr(m, "_call", lambda fn, dev, *args: calls.append((fn.__name__, args)))
    return calls


class Stand:
    """What the C form reads of a tensor, at an address that nobody reads."""
    device = "cuda:0"

    def __init__(self, shape, dtype, stride=None, ptr=1 << 20):
        n, packed = 1, []
        for s in reversed(shape):
            packed.insert(0, n)
            n *= max(s, 1)
        self.shape, self.dtype, self._stride, self._ptr = tuple(shape), dtype, tuple(stride or packed), ptr

    def stride(self):
        return self._stride

    def get_device(self):
        return 0

    def data_ptr(self):
        return self._ptr


class Refused(Exception):
    pass


@pytest.fixture
def c_form(m):
    """The C form with stand-ins for tensors.  The C entries run their checks, which must refuse the call: with a
    GPU at hand one that did not would launch on the stand-ins' addresses."""
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    m._plain()
    mod = m._marshal

    def check(rc):
        raise Refused(rc, m.lib().mla_last_error().decode())

    mod.init(Stand, lambda shape, dtype, device: Stand(shape, dtype), lambda: 0, lambda dev: 0, check, BF, U8, I8, F32, I32, I64)
    yield mod
    m._marshal = None       # set up again for tensors by the next use


# ------------------------------------------------------------------------------------------ rows that overlap

def test_python_form_hands_over_the_true_row_strides(m, python_form):
    B, T, k, cols, W = 4, 4, 8, 5, 40
    z = lambda *s, dt: torch.zeros(s, dtype=dt)
    q, w, c, s = z(T, 2, 128, dt=U8), z(T, 2, dt=F32), z(3, 16, 128, dt=U8), z(3, 16, dt=F32)
    table, lens = z(1, cols, dt=I32), z(B, dt=I32)
    one = lambda t: t.expand(B, -1)
    sc = z(1, W, dt=F32)

    def strides(name):
        (got, args), = python_form
        python_form.clear()
        at = {"mla_index_gather": (9,), "mla_index_scores": (14, 23), "mla_index_select": (1, 12, 14, 16),
              "mla_selected_decode": (10, 15)}[name]
        assert got == name
        return [args[i] for i in at]

    cu = z(B + 1, dt=I32)
    m.index_gather(c, s, one(table), cu, fmt="fp8", num_tokens=3)
    assert strides("mla_index_gather") == [0]
    m.index_scores(q, w, c, s, one(table), lens, fmt="fp8", max_context=W, scores=one(sc))
    assert strides("mla_index_scores") == [0, 0]
    m.index_select(one(sc), lens, k, block_table=one(table), page_size=16, num_blocks=3, blocks=one(z(1, k, dt=I32)),
                   slots=one(z(1, k, dt=I32)))
    assert strides("mla_index_select") == [0, 0, 0, 0]
    args = (z(T, 2, 576, dt=BF), z(3, 16, 576, dt=BF), one(table), lens, one(z(1, k, dt=I32)))
    m.selected_decode(*args, fmt="bf16", softmax_scale=1.0, workspace=z(1 << 16, dt=U8))
    assert strides("mla_selected_decode") == [0, 0]
    # overlapping rows with a stride of their own, and rows further apart than they are long
    far = lambda t, step: torch.as_strided(torch.zeros(step * T + t.shape[1], dtype=t.dtype), (T, t.shape[1]), (step, 1))
    m.index_select(far(sc, W - 1), lens, k, blocks=far(z(1, k, dt=I32), k + 3))
    assert strides("mla_index_select")[:2] == [W - 1, k + 3]


def test_python_form_of_a_single_row_hands_over_its_length(m, python_form):
    """The stride of one row means nothing."""
    row = lambda n, dt: torch.as_strided(torch.zeros(n, dtype=dt), (1, n), (1, 1))
    m.index_select(row(40, F32), torch.zeros(1, dtype=I32), 8, block_table=row(5, I32), page_size=16, num_blocks=3, blocks=row(8, I32),
                   slots=row(8, I32))
    (_, args), = python_form
    assert [args[i] for i in (1, 12, 14, 16)] == [40, 8, 8, 5]


def test_c_form_hands_over_the_true_row_strides(c_form):
    B, T, k, cols, W = 4, 4, 8, 5, 40
    table, lens, cu = Stand((B, cols), I32, (0, 1)), Stand((B,), I32), Stand((B + 1,), I32)
    good = Stand((B, cols), I32)
    c, s = Stand((3, 16, 128), U8), Stand((3, 16), F32)
    q, w = Stand((T, 2, 128), U8), Stand((T, 2), F32)

    def refused(name, message, *args):
        with pytest.raises(Refused, match=message) as e:
            getattr(c_form, name)(*args)
        assert e.value.args[0] == INVALID

    refused("gather", "block_table", c, s, table, cu, None, 1, 3, None)
    scores = lambda t, out: ("scores", "block_table" if t is table else "scores rows", q, w, c, s, t, lens, None, 1, 1, W, out)
    refused(*scores(table, None))
    refused(*scores(good, Stand((T, W), F32, (0, 1))))
    refused(*scores(good, Stand((T, W), F32, (W - 1, 1))))
    x, thin = Stand((T, W), F32), lambda n, dt: Stand((T, n), dt, (0, 1))

    def select(message, x=x, blocks=None, t=good, slots=None):
        refused("select", message, x, lens, k, None, 1, 0, 0, t, 16, 3, blocks, slots)

    select("scores rows", x=thin(W, F32))
    select("blocks rows", blocks=thin(k, I32))
    select("block_table", t=table)
    select("slots rows", slots=thin(k, I32))
    dec = lambda t, b: (Stand((T, 2, 576), BF), Stand((3, 16, 576), BF), t, lens, b, None, 0, 1.0, 1.0, 1.0, None, False, None, None)
    refused("selected", "blocks rows", *dec(good, thin(k, I32)))
    refused("selected", "block_table", *dec(table, Stand((T, k), I32)))


# ------------------------------------------------------------------------------------------ no columns

def test_selection_without_columns_needs_no_scores(m):
    """Width 0: the address of scores (and of a table of no columns) may be NULL.  The call is given a bad
    page size, which is looked at last, so that it is refused either way."""
    L, FAKE = m.lib(), 1 << 20
    select = lambda x, width, table: L.mla_index_select(x, width, width, FAKE, FAKE, 2, 3, 1, 8, 0, 0, FAKE, 8, FAKE, 8, table, 0, 0, 0, 0, None)
    assert select(None, 0, None) == INVALID and b"page_size" in L.mla_last_error()
    assert select(None, 5, FAKE) == INVALID and b"pointer" in L.mla_last_error()
    assert select(FAKE, 5, None) == INVALID and b"block_table" in L.mla_last_error()


# ------------------------------------------------------------------------------------------ caches of another format

KV = [("bf16", BF, 576, True), ("bf16", U8, 1152, True), ("fp8", U8, 576, True), ("fp8", I8, 640, True), ("fp8_ds_mla", U8, 656, True),
      ("fp8_ds_mla", U8, 1152, True), ("bf16", BF, 512, False), ("bf16", U8, 576, False), ("fp8", BF, 576, False), ("fp8", U8, 512, False),
      ("fp8_ds_mla", BF, 576, False), ("fp8_ds_mla", U8, 576, False), ("fp8_ds_mla", BF, 656, False)]


def decode_args(fmt, dtype, width, tensor):
    q = tensor((2, 4, 576), U8 if fmt == "fp8" else BF)
    return q, tensor((3, 16, width), dtype), tensor((2, 5), I32), tensor((2,), I32), tensor((2, 2), I32)


@pytest.mark.parametrize("fmt,dtype,width,fits", KV)
def test_python_form_refuses_a_cache_of_another_format(m, python_form, fmt, dtype, width, fits):
    args = decode_args(fmt, dtype, width, lambda shape, dt: torch.zeros(shape, dtype=dt))
    run = lambda: m.selected_decode(*args, fmt=fmt, softmax_scale=1.0, workspace=torch.zeros(1 << 16, dtype=U8))
    if fits:
        run()
        assert len(python_form) == 1
        return
    with pytest.raises((ValueError, TypeError), match="kv_cache"):
        run()
    assert not python_form


@pytest.mark.parametrize("fmt,dtype,width,fits", KV)
def test_c_form_declines_a_cache_of_another_format(c_form, fmt, dtype, width, fits):
    """One that fits reaches the C entry, which refuses the workspace here."""
    args = decode_args(fmt, dtype, width, Stand)
    number = {"bf16": 0, "fp8": 1, "fp8_ds_mla": 2}[fmt]
    run = lambda: c_form.selected(*args, None, number, 1.0, 1.0, 1.0, None, False, Stand((8,), U8, ptr=(1 << 20) + 8), None)
    if fits:
        with pytest.raises(Refused):
            run()
    else:
        assert run() is None


# ------------------------------------------------------------------------------------------ dimensions of one entry

def test_python_form_of_single_rows_and_heads(m, python_form):
    """A dimension of one entry is handed over with what the entry spans, whatever its stride (1 here, as of a
    transposed column)."""
    thin = lambda *shape, dt: torch.as_strided(torch.zeros(4096, dtype=dt), shape, tuple([1] * len(shape)))
    lens, cu = torch.zeros(1, dtype=I32), torch.zeros(2, dtype=I32)
    q, w, c, s = thin(1, 1, 128, dt=BF), thin(1, 1, dt=F32), thin(1, 1, 128, dt=BF), thin(1, 4, dt=F32)
    m.index_q_cache_insert(q, thin(1, 128, dt=BF), w, c, None, torch.zeros(1, dtype=I64), fmt="bf16")
    m.index_scores(q, w, c, None, thin(1, 3, dt=I32), lens, fmt="bf16", max_context=4)
    c8 = torch.as_strided(torch.zeros(4096, dtype=U8), (1, 4, 128), (1, 128, 1))
    m.index_gather(c8, s, thin(1, 3, dt=I32), cu, fmt="fp8", num_tokens=1, dst=thin(1, 128, dt=BF))
    m.selected_decode(thin(1, 1, 576, dt=BF), thin(1, 1, 576, dt=BF), thin(1, 3, dt=I32), lens, thin(1, 2, dt=I32), fmt="bf16",
                      softmax_scale=1.0, out=thin(1, 1, 520, dt=BF), workspace=torch.zeros(1 << 12, dtype=U8))
    insert, scores, gather, decode = [a for _, a in python_form]
    assert [insert[i] for i in (1, 2, 4, 6, 13, 14)] == [128, 128, 128, 1, 256, 256]
    assert [scores[i] for i in (1, 2, 4, 8, 9, 14)] == [128, 128, 1, 256, 256, 3]
    assert [gather[i] for i in (3, 4, 6, 9, 16)] == [512, 128, 4, 3, 128]
    assert [decode[i] for i in (1, 2, 6, 7, 10, 15, 24, 25)] == [576, 576, 1152, 1152, 3, 2, 520, 520]


def test_c_form_of_single_rows_and_heads(c_form):
    """The same: the only refusal is the one that each call is given, or that there is no device here."""
    thin = lambda *shape, dt: Stand(shape, dt, tuple([1] * len(shape)))
    lens = Stand((1,), I32)
    with pytest.raises(Refused, match="page_size"):
        c_form.select(thin(1, 9, dt=F32), lens, 4, None, 1, 0, 0, thin(1, 3, dt=I32), 0, 3, thin(1, 4, dt=I32), thin(1, 4, dt=I32))
    with pytest.raises(Refused, match="cudaGetDevice"):
        c_form.selected(thin(1, 1, 576, dt=BF), thin(1, 1, 576, dt=BF), thin(1, 3, dt=I32), lens, thin(1, 2, dt=I32), None, 0, 1.0, 1.0, 1.0,
                        thin(1, 1, 520, dt=BF), False, Stand((1 << 20,), U8, ptr=(1 << 20) + 8), None)
    q, c, s = thin(1, 1, 128, dt=BF), thin(1, 1, 128, dt=BF), thin(1, 9, dt=F32)
    with pytest.raises(Refused, match="must be given together"):
        c_form.insert(q, thin(1, 128, dt=BF), thin(1, 1, dt=F32), c, None, Stand((1,), I64), 0, 1.0, None, thin(1, 64, dt=F32), None, None)
    with pytest.raises(Refused, match="NULL"):
        c_form.gather(c, None, thin(1, 3, dt=I32), Stand((2,), I32, ptr=0), None, 0, 1, thin(1, 128, dt=BF))
    with pytest.raises(Refused, match="scores rows"):       # the last check: an odd address
        c_form.scores(q, thin(1, 1, dt=F32), c16(), None, thin(1, 3, dt=I32), lens, None, 0, 1, 9, Stand((1, 9), F32, (1, 1), ptr=(1 << 20) + 1))


def c16():
    return Stand((1, 16, 128), BF, (1, 128, 1))
