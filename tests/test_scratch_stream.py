"""The workspace that a decode call takes for itself belongs to the stream that the
call launches on, not to torch's current one: the allocator hands a dropped
tensor's bytes to the next one of its stream, which must come after the launch."""
import contextlib

import pytest
import torch

from paged_kv_cache_29_gb300 import _binding as pa
from test_library_cpu import _OnDevice

B, HQ, HKV, D, NB, BS = 2, 8, 2, 128, 8, 16
BF, U8, I32, I64, F32 = torch.bfloat16, torch.uint8, torch.int32, torch.int64, torch.float32


class _Stream:
    """Stands for torch.cuda.Stream."""

    def __init__(self, handle, index=0):
        self.cuda_stream, self.device = handle, torch.device("cuda", index)


class _OtherStream:
    """Another library's stream: a handle and nothing else."""

    def __init__(self, handle):
        self.cuda_stream = handle


def _t(shape, dtype=BF):
    return _OnDevice(shape, dtype, 0)


def _calls():
    """Each decode entry point of the binding, called without a workspace."""
    q, q4, out, out4 = _t((B, HQ, D)), _t((B, 2, HQ, D)), _t((B, HQ, D)), _t((B, 2, HQ, D))
    tables, lens, rows, slots = _t((B, 4), I32), _t((B,), I32), _t((B, HKV, D)), _t((B,), I64)
    kc, c8, c1 = _t((NB, HKV, BS, D)), _t((NB, HKV, BS, D), U8), _t((NB, HKV, BS, D), torch.int8)
    sc, c4, p4 = _t((NB, HKV, BS), F32), _t((NB, HKV, BS, D // 2), U8), _t((NB, HKV, BS, 2))
    err = _t((1,), I32)
    return {
        "pa_decode": lambda st: pa.pa_decode(q, kc, kc, tables, lens, 0.1, out, 64, stream=st),
        "pa_append_decode": lambda st: pa.pa_append_decode(rows, rows, slots, kc, kc, q, tables, lens, 0.1, out, 64, stream=st),
        "pa_decode_multi": lambda st: pa.pa_decode_multi(q4, kc, kc, tables, lens, 0.1, out4, 64, stream=st),
        "pa_decode_window": lambda st: pa.pa_decode_window(q, kc, kc, tables, lens, 0.1, 32, out, 64, stream=st),
        "pa_decode_fp8": lambda st: pa.pa_decode_fp8(q, c8, c8, tables, lens, 0.1, out, 64, stream=st),
        "pa_append_decode_fp8": lambda st: pa.pa_append_decode_fp8(rows, rows, slots, c8, c8, q, tables, lens, 0.1, out, 64, stream=st),
        "pa_decode_int8": lambda st: pa.pa_decode_int8(q, c1, c1, sc, sc, tables, lens, 0.1, out, 64, stream=st),
        "pa_append_decode_int8": lambda st: pa.pa_append_decode_int8(rows, rows, slots, c1, c1, sc, sc, q, tables, lens, 0.1, out, 64,
                                                                     stream=st),
        "pa_decode_int4": lambda st: pa.pa_decode_int4(q, c4, c4, p4, p4, tables, lens, 0.1, out, 64, stream=st),
        "pa_test_withhold_tile": lambda st: pa.pa_test_withhold_tile(q, kc, kc, tables, lens, 0.1, out, 64, 0, err, stream=st),
    }


NAMES = list(_calls())


@pytest.fixture
def taken(monkeypatch):
    """(stream, bytes) of every tensor made during a call; the library reports success."""
    seen, under = [], [None]
    scratch = _t((1 << 20,), U8)

    class Library:
        def __getattr__(self, name):
            return (lambda *a: 4096) if "workspace_size" in name else (lambda *a: pa.PA_OK)

    @contextlib.contextmanager
    def stream(st):
        assert isinstance(st, torch.cuda.Stream)      # torch.cuda.stream takes no other
        before, under[0] = under[0], st.cuda_stream
        yield
        under[0] = before

    def empty(n, dtype, device):
        seen.append((under[0], n))
        return scratch

    monkeypatch.setattr(pa, "lib", Library)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "Stream", _Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", _Stream)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: _Stream(0))
    monkeypatch.setattr(pa, "_raw_stream", lambda: 7)
    monkeypatch.setattr(pa, "_raw_stream_of", lambda dev: 7)

    def run(name, st):
        call = _calls()[name]
        with monkeypatch.context() as m:
            m.setattr(torch, "empty", empty)
            call(st)
        return seen

    return run


@pytest.mark.parametrize("name", NAMES)
def test_a_given_stream_owns_the_scratch(taken, name):
    assert taken(name, _Stream(99)) == [(99, 4096)]


@pytest.mark.parametrize("name", NAMES)
def test_a_raw_handle_owns_the_scratch(taken, name):
    assert taken(name, 55) == [(55, 4096)]


@pytest.mark.parametrize("handle", [77, 0])
@pytest.mark.parametrize("name", NAMES)
def test_another_library_s_stream_owns_the_scratch(taken, name, handle):
    assert taken(name, _OtherStream(handle)) == [(handle, 4096)]


@pytest.mark.parametrize("name", NAMES)
def test_the_default_stream_s_handle_owns_the_scratch(taken, name):
    assert taken(name, 0) == [(0, 4096)]


@pytest.mark.parametrize("name", NAMES)
def test_without_a_stream_the_current_one_owns_it(taken, name):
    assert taken(name, None) == [(None, 4096)]


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_another_device_is_refused_before_anything_is_taken(taken, name):
    with pytest.raises(ValueError, match="stream belongs"):
        taken(name, _Stream(99, index=1))


def test_every_entry_point_that_takes_a_workspace_is_here():
    import inspect
    have = {n for n, f in vars(pa).items() if inspect.isfunction(f) and "workspace" in inspect.signature(f).parameters}
    assert have == set(NAMES)
