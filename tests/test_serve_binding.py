"""What the serving wrappers hand to the library (CPU only).

The library is replaced by a recorder, and the tensors say that they live on
a GPU, so that a call goes through its checks and to its end without one."""
import pytest

torch = pytest.importorskip("torch")


class Gpu(torch.Tensor):
    """A host tensor whose checks see one of device `index`."""

    index = 0
    is_cuda = True

    def get_device(self):
        return self.index


def gpu(t):
    return t.as_subclass(Gpu)


class Stream:
    cuda_stream = 0x51


class Recorder:
    """Stands for the library: notes the last call's arguments."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0

        return call


@pytest.fixture
def rec(monkeypatch):
    from gptq_post_weight_gb300 import _lib

    r = Recorder()
    monkeypatch.setattr(_lib, "_lib", r)
    monkeypatch.setattr(_lib, "_attention_ws", {})
    monkeypatch.setitem(_lib._serve_words, 0, (None, 0x77))
    _lib._serving()
    monkeypatch.setitem(_lib._serve, "current", lambda: 0)
    return r


def weights(rows, n):
    return (gpu(torch.zeros(rows * n // 2, dtype=torch.uint8)), gpu(torch.zeros(rows * n // 32, dtype=torch.uint8)),
            gpu(torch.zeros(rows, 32)))


def b16(*shape):
    return gpu(torch.zeros(*shape, dtype=torch.bfloat16))


# q4tp_linear's arguments at the library
X, LDX, TOKENS, BIAS, RESIDUAL, LDR, Y, LDY = 1, 2, 3, 9, 11, 12, 13, 14


@pytest.mark.parametrize("bias", [False, True])
def test_linear_refuses_rows_of_x_that_overlap(rec, bias):
    from gptq_post_weight_gb300 import _lib

    t, rows, n = 4, 6, 64
    b = b16(rows) if bias else None
    out = b16(t, rows + 2)[:, :rows]
    flat = b16(n + 8 * (t - 1))
    for x in (b16(1, n).expand(t, n), torch.as_strided(flat, (t, n), (8, 1))):
        with pytest.raises(ValueError, match="x must have rows that do not overlap"):
            _lib.q4tp_linear(x, *weights(rows, n), bias=b, out=out, stream=Stream)
    assert not rec.calls


def test_linear_hands_on_every_argument(rec):
    from gptq_post_weight_gb300 import _lib

    t, rows, n = 4, 6, 64
    x, b, r, out = b16(t, n + 8)[:, :n], b16(rows), b16(t, rows + 3)[:, :rows], b16(t, rows + 2)[:, :rows]
    _lib.q4tp_linear(x, *weights(rows, n), bias=b, act="silu", residual=r, out=out, stream=Stream)
    # No rows, in strides that the quick look at the arguments does not know.
    none = torch.as_strided(b16(2 * n), (0, n), (n, 2))
    _lib.q4tp_linear(none, *weights(rows, n), bias=b, residual=r[:0], out=out[:0], stream=Stream)
    (name, a), (_, e) = rec.calls
    assert name == "gptq_q4tp_linear"
    assert (a[X], a[LDX], a[TOKENS]) == (x.data_ptr(), n + 8, t)
    assert (a[BIAS], a[RESIDUAL], a[LDR], a[Y], a[LDY]) == (b.data_ptr(), r.data_ptr(), rows + 3, out.data_ptr(), rows + 2)
    assert e[TOKENS] == 0 and e[BIAS] == b.data_ptr() and e[RESIDUAL] is not None and e[LDY] >= rows


# kv4_attention's arguments at the library, and those of its workspace's size
Q_TS, TQ, Q_STARTS, SEQS, MAX_Q, SINGLE = 2, 4, 14, 15, 16, 5


@pytest.mark.parametrize("tq,heads,group,ts", [(9, 1, 1, 64), (0, 2, 2, 256), (0, 1, 1, 64), (1, 2, 2, 259),
                                               (1, 1, 1, 67), (9, 2, 2, 256)])
def test_attention_hands_on_q_starts(rec, tq, heads, group, ts):
    # One query head, no rows, a token stride that one token does not use.
    from gptq_post_weight_gb300 import _lib

    dim, page = 64, 16
    hq = heads * group
    q = torch.as_strided(b16(max(1, tq) * ts + hq * dim), (tq, hq, dim), (ts, dim, 1))
    cache = gpu(torch.zeros(4, heads, page * dim * 5 // 4, dtype=torch.uint8))
    table, lens = gpu(torch.zeros(2, 3, dtype=torch.int32)), gpu(torch.ones(2, dtype=torch.int32))
    starts = gpu(torch.tensor([0, 0, tq], dtype=torch.int32))
    _lib.kv4_attention(q, cache, table, lens, page, q_starts=starts, max_q=9, out=b16(tq, hq, dim), stream=Stream)
    (size, s), (name, a) = rec.calls
    assert (size, name) == ("gptq_kv4_attention_call_bytes", "gptq_kv4_attention")
    assert not s[SINGLE]
    assert (a[TQ], a[Q_STARTS], a[SEQS], a[MAX_Q]) == (tq, starts.data_ptr(), 2, 9)
    assert a[Q_TS] % 8 == 0 and (tq <= 1 or a[Q_TS] == ts)


def calls(stream=Stream):
    """One good call of each wrapper, its buffers given."""
    from gptq_post_weight_gb300 import _lib

    cache = gpu(torch.zeros(4, 2, 16 * 64 * 5 // 4, dtype=torch.uint8))
    k, slots = b16(3, 2, 64), gpu(torch.zeros(3, dtype=torch.int64))
    table, lens = gpu(torch.zeros(3, 1, dtype=torch.int32)), gpu(torch.ones(3, dtype=torch.int32))
    return {
        "x": lambda: _lib.q4tp_linear(b16(3, 64), *weights(6, 64), out=b16(3, 6), stream=stream),
        "k": lambda: _lib.kv4_write(cache, k, k, slots, 16, stream=stream),
        "cache": lambda: _lib.kv4_read(cache, slots, 64, 16, torch.bfloat16, stream=stream),
        "q": lambda: _lib.kv4_attention(b16(3, 4, 64), cache, table, lens, 16, out=b16(3, 4, 64), stream=stream),
    }


@pytest.fixture
def no_streams(monkeypatch):
    """torch.cuda.stream takes any object (kv4_read allocates under the call's)."""
    import contextlib

    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())


@pytest.mark.parametrize("name", ["x", "k", "cache", "q"])
def test_tensors_of_another_device_than_the_current_one_are_refused(rec, no_streams, monkeypatch, name):
    # The default stream has the same handle on every device: the launch would
    # run on the current one with the other one's addresses.
    from gptq_post_weight_gb300 import _lib

    calls()[name]()
    assert rec.calls
    monkeypatch.setitem(_lib._serve, "current", lambda: 1)
    rec.calls.clear()
    with pytest.raises(ValueError, match=f"{name} is on cuda:0, the current device is cuda:1"):
        calls()[name]()
    assert not rec.calls


@pytest.mark.parametrize("name", ["x", "k", "cache", "q"])
def test_streams_of_another_device_are_refused(rec, no_streams, name):
    class Other(Stream):
        device = torch.device("cuda", 1)

    with pytest.raises(ValueError, match="the stream is on cuda:1, the call's data on cuda:0"):
        calls(Other)[name]()
    assert not [c for c in rec.calls if not c[0].endswith("_bytes")]


def test_the_workspace_of_a_shape_is_the_device_s_own(rec, monkeypatch):
    from gptq_post_weight_gb300 import _lib

    calls()["q"]()
    monkeypatch.setattr(Gpu, "index", 1)
    monkeypatch.setitem(_lib._serve, "current", lambda: 1)
    monkeypatch.setitem(_lib._serve_words, 1, (None, 0x78))
    calls()["q"]()
    assert [c[0] for c in rec.calls].count("gptq_kv4_attention_call_bytes") == 2


def test_the_library_is_loaded_before_a_wrapper_finds_what_it_needs(monkeypatch):
    # Another thread's first call goes past `_serve or _serving()` as soon as
    # _serve holds anything, and then uses the library.
    from gptq_post_weight_gb300 import _lib

    seen = []
    monkeypatch.setattr(_lib, "_serve", {})
    monkeypatch.setattr(_lib, "load", lambda: seen.append(dict(_lib._serve)))
    assert _lib._serving() is _lib._serve and seen == [{}]


def test_threads_share_one_status_word(monkeypatch):
    import threading
    import time

    from gptq_post_weight_gb300 import _lib

    zeros = torch.zeros

    def slow(*a, **k):
        time.sleep(0.05)
        return zeros(4, dtype=torch.int32)

    monkeypatch.setattr(_lib, "_serve_words", {})
    monkeypatch.setattr(torch, "zeros", slow)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda i: type("S", (), {"synchronize": lambda self: None})())
    got, start = [], threading.Barrier(4)

    def first():
        start.wait()
        got.append(_lib._serve_word(0))

    threads = [threading.Thread(target=first) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert set(got) == {_lib._serve_words[0][1]} and len(got) == 4


@pytest.mark.parametrize("which", ["x", "bias", "residual", "q"])
def test_inputs_that_want_a_gradient_are_refused(rec, which):
    # The operators have no backward pass: the result would have no history,
    # and training would go on without that gradient.
    from gptq_post_weight_gb300 import _lib

    x, bias, residual, q = b16(3, 64), b16(6), b16(3, 6), b16(3, 4, 64)
    cache = gpu(torch.zeros(4, 2, 16 * 64 * 5 // 4, dtype=torch.uint8))
    table, lens = gpu(torch.zeros(3, 1, dtype=torch.int32)), gpu(torch.ones(3, dtype=torch.int32))
    dict(x=x, bias=bias, residual=residual, q=q)[which].requires_grad_()

    def call():
        if which == "q":
            _lib.kv4_attention(q, cache, table, lens, 16, out=b16(3, 4, 64), stream=Stream)
        else:
            _lib.q4tp_linear(x, *weights(6, 64), bias=bias, residual=residual, out=b16(3, 6), stream=Stream)

    with pytest.raises(ValueError, match=f"{which} requires a gradient"):
        call()
    assert not rec.calls
    with torch.no_grad():
        call()
    assert rec.calls
