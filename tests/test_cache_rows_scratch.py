"""The workspaces that the calls which say what rows of a cache count take for themselves
belong to the stream that the call launches on, as the decode calls' do."""
import inspect

import pytest

import test_scratch_stream as scratch
from paged_kv_cache_29_gb300 import _binding_rows as rows
from test_scratch_stream import B, BS, D, F32, HKV, HQ, I32, NB, _OtherStream, _Stream, _t, taken  # noqa: F401


def calls():
    q, out, kc = _t((B, HQ, D)), _t((B, HQ, D)), _t((NB, HKV, BS, D))
    tables, lens, w = _t((B, 4), I32), _t((B,), I32), _t((NB, HKV, BS), F32)
    return {
        "pa_decode_sinks": lambda st: rows.pa_decode_sinks(q, kc, kc, tables, lens, 0.1, 32, 4, out, 64, stream=st),
        "pa_decode_weights": lambda st: rows.pa_decode_weights(q, kc, kc, tables, lens, 0.1, out, w, 64, stream=st),
        "pa_evict": lambda st: rows.pa_evict(kc, kc, w, tables, lens, lens, tables, lens, 64, stream=st),
    }


@pytest.mark.parametrize("stream,owner", [(_Stream(99), 99), (55, 55), (_OtherStream(77), 77), (_OtherStream(0), 0), (0, 0), (None, None)])
@pytest.mark.parametrize("name", list(calls()))
def test_the_launching_stream_owns_the_scratch(taken, monkeypatch, name, stream, owner):  # noqa: F811
    monkeypatch.setattr(scratch, "_calls", calls)
    assert taken(name, stream) == [(owner, 4096)]


@pytest.mark.parametrize("name", list(calls()))
def test_a_stream_of_another_device_is_refused_before_anything_is_taken(taken, monkeypatch, name):  # noqa: F811
    monkeypatch.setattr(scratch, "_calls", calls)
    with pytest.raises(ValueError, match="stream belongs"):
        taken(name, _Stream(99, index=1))


def test_every_call_that_takes_a_workspace_is_here():
    have = {n for n, f in vars(rows).items() if inspect.isfunction(f) and "workspace" in inspect.signature(f).parameters}
    assert have == set(calls())
