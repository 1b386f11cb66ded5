"""The calls that say which rows of a cache count, without a GPU: what they refuse, the
workspaces they ask for, the references themselves, and the block manager's side."""
import numpy as np
import pytest

import cache_rows_reference as ref
from paged_kv_cache_29_gb300 import _binding as pa
from paged_kv_cache_29_gb300 import build as build_mod
from paged_kv_cache_29_gb300.block_manager import BlockManager, OutOfBlocks

P = 1 << 20                     # never dereferenced: every call below fails validation first
INVALID, UNSUPPORTED, WORKSPACE = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED, pa.PA_ERR_WORKSPACE
HUGE = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return pa.lib()


SIZES = dict(B=4, Q=1, Hq=8, Hkv=2, D=128, bs=16, NB=10, mb=4, mcl=64, dtype=1, ws=None, wsb=0, err=None)


def sinks(lib, **kw):
    a = dict(q=P, k=P, v=P, bt=P, cl=P, scale=0.1, window=16, first=4, out=P, **SIZES)
    a.update(kw)
    return lib.pa_decode_sinks(*a.values(), None)


def weights(lib, **kw):
    a = dict(q=P, k=P, v=P, bt=P, cl=P, scale=0.1, out=P, rw=P, **SIZES)
    a.update(kw)
    return lib.pa_decode_weights(*a.values(), None)


def evict(lib, **kw):
    a = dict(k=P, v=P, kp=None, vp=None, rw=P, bt=P, cl=P, keep=P, to=P, out=P, first=4, last=4, B=4, Hkv=2, D=128, bs=16, NB=10, mb=4,
             mcl=64, dtype=1, ws=None, wsb=0, err=None)
    a.update(kw)
    return lib.pa_evict(*a.values(), None)


def verify(lib, **kw):
    a = dict(t=P, ts=100, tr=50, d=P, ds=100, dr=50, x=P, nd=None, u=P, out=P, acc=P, cl=None, lo=None, B=4, Q=4, V=1000, err=None)
    a.update(kw)
    return lib.pa_verify_draft(*a.values(), None)


@pytest.mark.parametrize("call", [sinks, weights])
@pytest.mark.parametrize("kw,status", [
    (dict(), WORKSPACE), (dict(B=0, q=None), pa.PA_OK), (dict(B=-1), INVALID), (dict(Q=0), INVALID), (dict(Q=9), INVALID),
    (dict(Hq=7), INVALID), (dict(Hkv=0), INVALID), (dict(D=0), INVALID), (dict(D=257), UNSUPPORTED), (dict(bs=0), INVALID), (dict(NB=0), INVALID),
    (dict(mcl=65), INVALID), (dict(mcl=-1), INVALID), (dict(mb=-1), INVALID), (dict(dtype=2), INVALID), (dict(dtype=7), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(q=None), INVALID), (dict(out=None), INVALID),
    (dict(bt=None), INVALID), (dict(cl=None), INVALID), (dict(k=P + 8), INVALID), (dict(q=P + 2), INVALID), (dict(bt=P + 2), INVALID),
    (dict(Hq=1 << 21, Hkv=1 << 21), UNSUPPORTED), (dict(Hq=2048, Hkv=1), UNSUPPORTED), (dict(Hq=1024, Hkv=1, Q=2), UNSUPPORTED),
    (dict(mcl=HUGE, mb=HUGE), UNSUPPORTED), (dict(B=HUGE, Hq=1 << 18, Hkv=1 << 18), UNSUPPORTED),
])
def test_decode_calls_refuse(lib, call, kw, status):
    assert call(lib, **kw) == status


def test_what_one_of_the_two_refuses(lib):
    assert sinks(lib, window=0) == INVALID and sinks(lib, window=-3) == INVALID and sinks(lib, first=-1) == INVALID
    assert sinks(lib, window=HUGE, first=HUGE) == WORKSPACE
    assert weights(lib, rw=None) == INVALID and weights(lib, rw=P + 2) == INVALID


@pytest.mark.parametrize("B,Q,hq,D,mcl", [(4, 1, 8, 128, 64), (128, 2, 32, 128, 8192), (1, 1, 1, 64, 513), (5000, 1, 3, 7, 600), (3, 1, 5, 33, 1537)])
def test_workspaces(lib, B, Q, hq, D, mcl):
    need = lib.pa_decode_workspace_size_weights(B, Q, hq, D, mcl)
    seqs, parts = min(B, 4096), max(1, -(-mcl // 512))
    units = seqs * hq * parts
    base = 256 + 16 * units + 8 * units * Q + (4 * units * Q * D if parts > 1 else 0)
    states = -(-8 * seqs * hq * Q // 16) * 16
    assert need == -(-base // 16) * 16 + states + 4 * seqs * hq * Q * (-(-mcl // 16) * 16)
    mb = -(-mcl // 16)
    sizes = dict(B=B, Q=Q, Hq=hq, Hkv=1, D=D, mcl=mcl, mb=mb)
    assert weights(lib, **sizes, ws=P, wsb=need - 1) == WORKSPACE and weights(lib, **sizes, ws=P + 8, wsb=need) == WORKSPACE
    need = lib.pa_decode_workspace_size_multi(B, Q, hq, D, mcl)
    assert sinks(lib, **sizes, ws=P, wsb=need - 1) == WORKSPACE and sinks(lib, **sizes, ws=P + 8, wsb=need) == WORKSPACE
    need = lib.pa_evict_workspace_size(B, hq, mcl)
    assert need == 8 * B * hq * mcl + 4 * (B * hq + 2 * B)
    assert evict(lib, B=B, Hkv=hq, mcl=mcl, mb=mb, ws=P, wsb=need - 1) == WORKSPACE
    assert lib.pa_decode_workspace_size_weights(0, Q, hq, D, mcl) == 0 and lib.pa_evict_workspace_size(0, hq, mcl) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(), WORKSPACE), (dict(B=0, k=None), pa.PA_OK), (dict(B=-1), INVALID), (dict(first=-1), INVALID), (dict(last=-1), INVALID),
    (dict(Hkv=0), INVALID), (dict(D=0), INVALID), (dict(bs=0), INVALID), (dict(NB=0), INVALID), (dict(mcl=65), INVALID), (dict(dtype=5), INVALID),
    (dict(dtype=-1), INVALID), (dict(D=4), UNSUPPORTED), (dict(D=512, dtype=0), UNSUPPORTED), (dict(D=8, dtype=2), UNSUPPORTED),
    (dict(D=33, dtype=4, kp=P, vp=P), UNSUPPORTED), (dict(NB=1 << 24, bs=256), UNSUPPORTED), (dict(Hkv=1 << 21), UNSUPPORTED),
    (dict(B=1 << 23), UNSUPPORTED), (dict(k=None), INVALID), (dict(rw=None), INVALID), (dict(keep=None), INVALID), (dict(to=None), INVALID),
    (dict(out=None), INVALID), (dict(kp=P, vp=P), INVALID), (dict(dtype=3), INVALID), (dict(dtype=3, kp=P), INVALID),
    (dict(dtype=3, kp=P, vp=P), WORKSPACE), (dict(dtype=4, kp=P, vp=P + 2), INVALID), (dict(dtype=4, kp=P, vp=P), WORKSPACE),
    (dict(v=P + 8), INVALID), (dict(cl=P + 1), INVALID), (dict(dtype=2), WORKSPACE), (dict(dtype=0), WORKSPACE),
])
def test_evict_refuses(lib, kw, status):
    assert evict(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(B=0, t=None), pa.PA_OK), (dict(B=-1), INVALID), (dict(Q=-1), INVALID), (dict(V=0), INVALID), (dict(cl=P), INVALID), (dict(lo=P), INVALID),
    (dict(Q=65), UNSUPPORTED), (dict(V=(1 << 22) + 1), UNSUPPORTED), (dict(B=1 << 25), UNSUPPORTED), (dict(t=None), INVALID), (dict(u=None), INVALID),
    (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(acc=None), INVALID), (dict(t=P + 2), INVALID), (dict(u=P + 1), INVALID),
])
def test_verify_refuses(lib, kw, status):
    assert verify(lib, **kw) == status


def test_references():
    """The plain references on cases small enough to write out."""
    assert list(ref.visible(10, 1, 0, 3, 2)) == [0, 1, 7, 8, 9]
    assert list(ref.visible(10, 2, 0, 3, 2)) == [0, 1, 6, 7, 8]
    assert list(ref.visible(4, 1, 0, 3, 3)) == [0, 1, 2, 3]
    assert list(ref.visible(3, 2, 1, 0, 0)) == [0, 1, 2]
    w = np.array([0.0, 5.0, 1.0, 5.0, np.nan, 5.0, -1.0, 9.0])
    assert ref.kept_rows(w, 8, 4, 1, 1) == [0, 1, 3, 7]
    assert ref.kept_rows(w, 8, 2, 0, 0) == [1, 7] and ref.kept_rows(w, 8, 9, 0, 0) == list(range(8))
    assert ref.kept_rows(w, 8, 7, 0, 0) == [0, 1, 2, 3, 5, 6, 7]
    k = np.array([[[1.0, 0.0]], [[0.0, 1.0]]])
    out, weight, _, _ = ref.attention(np.array([[[np.log(3.0), 0.0]]]), k, k, 1.0, 1)
    assert np.allclose(out[0, 0], [0.75, 0.25]) and np.allclose(weight[:, 0], [0.75, 0.25])
    p, q = np.float32([[0.5, 0.5], [0.25, 0.75]]), np.float32([[1.0, 0.0]])
    assert ref.verify(p, q, [0], [0.4, 0.5], 1)[:2] == (1, 1)
    assert ref.verify(p, q, [0], [0.6, 0.5], 1)[:2] == (0, 1)
    assert ref.verify(p, None, [1], [0.6, 0.9], 1)[:2] == (0, 0)


# ------------------------------------------------------------ block manager


def test_truncate_takes_rejected_tokens_back():
    m = BlockManager(8, 4)
    m.admit("a", range(6))
    for t in (6, 7, 8, 9):
        m.append("a", t)
    assert m.num_tokens("a") == 10 and len(m.block_table("a")) == 3
    assert m.truncate("a", 7) is None                  # the second block was full and had a key
    m.check()
    assert m.num_tokens("a") == 7 and len(m.block_table("a")) == 2
    m.append("a", 99)                                  # full again, with another token
    assert m.admit("b", [0, 1, 2, 3, 4, 5, 6, 7]) == 4  # the old second block is not found
    assert m.admit("c", [0, 1, 2, 3, 4, 5, 6, 99]) == 8
    m.check()
    assert m.truncate("a", 0) is None and m.num_tokens("a") == 0
    m.append("a", 1)
    m.check()
    with pytest.raises(ValueError):
        m.truncate("a", 2)
    with pytest.raises(ValueError):
        m.truncate("a", -1)


def test_truncate_into_a_shared_block_copies_it():
    m = BlockManager(4, 4)
    m.admit("a", range(7))
    m.fork("a", "b")
    pair = m.truncate("a", 5)
    assert pair is not None and pair[0] == m.block_table("b")[1] and pair[1] == m.block_table("a")[1]
    assert m.num_tokens("a") == 5 and m.num_tokens("b") == 7
    m.check()
    assert m.truncate("b", 4) is None                  # at a block's end: nothing is cut
    m.check()
    m = BlockManager(2, 4)
    m.admit("a", range(7))
    m.fork("a", "b")
    with pytest.raises(OutOfBlocks):
        m.truncate("a", 5)
    assert m.num_tokens("a") == 7
    m.check()


def test_evict_keeps_private_blocks_and_replaces_shared_ones():
    m = BlockManager(12, 4)
    m.admit("a", range(14))
    m.fork("a", "b")
    for t in range(5):
        m.append("a", t)                               # copy-on-write of the last, then blocks of its own
    before = {s: m.block_table(s) for s in "ab"}
    out = m.evict({"a": 17, "b": 9})
    m.check()
    for s, n in (("a", 17), ("b", 9)):
        assert m.block_table(s) == out[s] and m.num_tokens(s) == n and len(out[s]) == -(-n // 4)
    held = set(before["a"]) | set(before["b"])
    for s in "ab":
        for i, b in enumerate(out[s]):
            assert b == before[s][i] or b not in held
    assert [out["a"][i] == before["a"][i] for i in range(5)] == [False, False, False, True, True]
    assert len(set(out["a"] + out["b"])) == len(out["a"]) + len(out["b"])
    assert m.append("a", 1).slot == out["a"][4] * 4 + 1


def test_evicted_rows_are_not_found_as_a_prefix():
    m = BlockManager(8, 4)
    m.admit("a", range(8))
    assert m.evict({"a": 4})["a"] == m.block_table("a")
    for t in range(4):
        m.append("a", t)
    assert m.admit("b", range(8)) == 0
    m.fork("a", "c")
    m.release("a")
    for t in range(5):
        m.append("c", t)
    m.release("b")
    m.release("c")
    assert m.admit("d", range(8)) == 8                 # b's own blocks, whose tokens are known
    m.check()
    with pytest.raises(ValueError):
        m.evict({"d": 9})
    m.fork("d", "e")
    m.admit("f", [50] * 24)
    with pytest.raises(OutOfBlocks):
        m.evict({"d": 5, "e": 5})
    m.check()
    assert m.num_tokens("d") == 8
