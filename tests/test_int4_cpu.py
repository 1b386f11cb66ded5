"""The 4-bit cache and norm and rotation calls without a GPU: the reference that
the GPU tests use, and the arguments that the library and the binding refuse
before anything is enqueued."""
import ctypes
import dataclasses

import numpy as np
import pytest
import torch

import rows_reference as ref
from paged_kv_cache_29_gb300 import _binding as pa
from paged_kv_cache_29_gb300 import build as build_mod
from test_library_cpu import FAKE, _OnDevice

INVALID, UNSUPPORTED, WORKSPACE = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED, pa.PA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return pa.lib()


# ------------------------------------------------------------- the reference


def test_pair_covers_the_row_and_codes_are_within_half_a_step():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((400, 64)) * 10.0 ** rng.uniform(-4, 4, (400, 1)) + rng.uniform(-3, 3, (400, 1))).astype(np.float32)
    packed, pairs = ref.quantise4(x)
    lo, s = ref.bf16_value(pairs[:, 0]).astype(np.float64), ref.bf16_value(pairs[:, 1]).astype(np.float64)
    assert (lo <= x.min(-1)).all() and (lo + 15 * s >= x.max(-1) * (1 - 2.0 ** -22) - 2.0 ** -22 * np.abs(lo)).all()
    err = np.abs(ref.values4(packed, pairs) - x)
    assert (err <= s[:, None] / 2 + 2.0 ** -22 * (np.abs(x) + np.abs(lo[:, None]))).all()


def test_directed_rounding_of_the_pair():
    x = np.array([1.0, 1.0 + 2.0 ** -8, -1.0 - 2.0 ** -8, 0.0, 2.0 ** -133], np.float32)
    assert ref.bf16_value(ref.bf16_bits(x, "down")).tolist() == [1.0, 1.0, -1.0 - 2.0 ** -7, 0.0, 2.0 ** -133]
    assert ref.bf16_value(ref.bf16_bits(x, "up")).tolist() == [1.0, 1.0 + 2.0 ** -7, -1.0, 0.0, 2.0 ** -133]


def test_constant_row_is_exact():
    packed, pairs = ref.quantise4(np.full((1, 32), -2.5, np.float32))
    assert not packed.any() and ref.values4(packed, pairs).tolist() == [[-2.5] * 32]


def test_reference_attention_sees_what_the_masks_leave():
    """With V rows that name their row, a window of one gives each token its own row."""
    n, D, Q = 20, 32, 3
    x = np.broadcast_to(np.arange(32, dtype=np.float32)[:, None], (32, D)).reshape(2, 16, 1, D).transpose(0, 2, 1, 3)
    kc, kp = ref.quantise4(np.random.default_rng(1).standard_normal((2, 1, 16, D)).astype(np.float32))
    vc, vp = ref.quantise4(np.ascontiguousarray(x))
    out, _ = ref.attention4(np.ones((Q, 1, D)), (kc, vc, kp, vp), [0, 1], n, 0.1, 16, window=1)
    assert out[:, 0, 0].tolist() == [17.0, 18.0, 19.0]


def test_reference_rotation_keeps_lengths():
    rng = np.random.default_rng(2)
    angle = rng.uniform(0, 6, (50, 8))
    cs = np.concatenate([np.cos(angle), np.sin(angle)], 1)
    x = rng.standard_normal((5, 2, 32))
    for inter in (False, True):
        y, _ = ref.norm_rope(x, None, rng.integers(0, 50, (2, 5)), cs, interleaved=inter, pair_axis=[0, 1] * 4)
        np.testing.assert_allclose((y ** 2).sum(-1), (x ** 2).sum(-1))


# ------------------------------------------------------------------ refusals


def _append(lib, **kw):
    a = dict(k=FAKE, v=FAKE, dtype=1, slots=FAKE, kc=FAKE, vc=FAKE, kp=FAKE, vp=FAKE, T=4, hkv=2, d=128, bs=16, nb=8)
    a.update(kw)
    return lib.pa_reshape_and_cache_int4(*a.values(), None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INVALID), (dict(kp=None), INVALID), (dict(vp=FAKE + 4), INVALID), (dict(v=FAKE + 8), INVALID),
    (dict(slots=FAKE + 4), INVALID), (dict(dtype=2), INVALID), (dict(T=-1), INVALID), (dict(bs=0), INVALID),
    (dict(nb=0), INVALID), (dict(d=48), UNSUPPORTED), (dict(d=288), UNSUPPORTED), (dict(T=0, k=None), pa.PA_OK),
])
def test_append_refusals(lib, kw, status):
    assert _append(lib, **kw) == status


def _gather(lib, **kw):
    a = dict(kc=FAKE, vc=FAKE, kp=FAKE, vp=FAKE, bt=FAKE, cl=FAKE, rs=FAKE, ko=FAKE, vo=FAKE, dtype=1, rows=100, B=2, hkv=2,
             d=128, bs=16, nb=8, mb=4, mcl=64)
    a.update(kw)
    return lib.pa_gather_int4(*a.values(), None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(kc=None), INVALID), (dict(ko=None), INVALID), (dict(rs=FAKE + 4), INVALID), (dict(vo=FAKE + 8), INVALID),
    (dict(dtype=3), INVALID), (dict(rows=-1), INVALID), (dict(mcl=65), INVALID), (dict(B=-1), INVALID),
    (dict(d=16), UNSUPPORTED), (dict(d=512), UNSUPPORTED), (dict(B=0, bt=None), pa.PA_OK),
])
def test_gather_refusals(lib, kw, status):
    assert _gather(lib, **kw) == status


def _decode(lib, **kw):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, kp=FAKE, vp=FAKE, bt=FAKE, cl=FAKE, scale=0.1, window=0, out=FAKE, B=4, Q=1, hq=8, hkv=2,
             d=128, bs=16, nb=10, mb=40, mcl=64, ws=None, wsb=0)
    a.update(kw)
    return lib.pa_decode_int4(*a.values(), None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(kp=None), INVALID), (dict(vc=FAKE + 8), INVALID), (dict(bt=FAKE + 2), INVALID),
    (dict(hq=6, hkv=4), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(window=-1), INVALID), (dict(Q=0), INVALID), (dict(mcl=641), INVALID), (dict(B=-1), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(bs=8), UNSUPPORTED), (dict(hq=18, hkv=2), UNSUPPORTED),
    (dict(Q=3), UNSUPPORTED), (dict(mcl=2 ** 31 - 16, mb=2 ** 27), UNSUPPORTED), (dict(nb=2 ** 31 - 1, hkv=4), UNSUPPORTED),
    (dict(B=0, q=None), pa.PA_OK), (dict(), WORKSPACE), (dict(ws=FAKE, wsb=100), WORKSPACE),
    (dict(ws=FAKE + 8, wsb=1 << 30), WORKSPACE),
])
def test_decode_refusals(lib, kw, status):
    assert _decode(lib, **kw) == status


def test_decode_workspace_is_the_multi_query_size(lib):
    for B, Q, hq, d, mcl in [(4, 2, 8, 128, 600), (5000, 1, 8, 64, 2000)]:
        need = lib.pa_decode_workspace_size_multi(B, Q, hq, d, mcl)
        kw = dict(B=B, Q=Q, hq=hq, d=d, mcl=mcl, mb=200, ws=FAKE)
        assert _decode(lib, **kw, wsb=need - 1) == WORKSPACE


NORM = dict(q=FAKE, k=FAKE, q_stride=1024, k_stride=256, q_out=FAKE, q_out_stride=1024, q_weight=FAKE, k_weight=FAKE, eps=1e-6,
            weight_offset=0.0, cos_sin=FAKE, positions=FAKE, pair_axis=None, num_tokens=4, num_heads=8, num_kv_heads=2,
            head_dim=128, rot_dim=128, max_position=10, num_axes=1, interleaved=0, dtype=1, weight_dtype=1)


def _norm(lib, k_out=FAKE, k_out_stride=256, **kw):
    args = pa._NormRopeArgs(**{**NORM, **kw})
    return lib.pa_norm_rope(ctypes.byref(args), k_out, k_out_stride, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(q=FAKE + 8), INVALID), (dict(q_out=None), INVALID), (dict(k_out=None), INVALID),
    (dict(k_out_stride=128), INVALID), (dict(q_stride=1000), INVALID), (dict(q_stride=1028), INVALID),
    (dict(k_stride=128), INVALID), (dict(q_weight=FAKE + 4), INVALID), (dict(cos_sin=None), INVALID),
    (dict(positions=None), INVALID), (dict(positions=FAKE + 2), INVALID), (dict(max_position=0), INVALID),
    (dict(num_axes=0), INVALID), (dict(num_axes=5), INVALID), (dict(pair_axis=bytes([0, 1] * 32)), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(weight_offset=float("inf")), INVALID),
    (dict(dtype=2), INVALID), (dict(weight_dtype=4), INVALID), (dict(rot_dim=144), INVALID), (dict(rot_dim=-16), INVALID),
    (dict(rot_dim=24), UNSUPPORTED), (dict(head_dim=40, rot_dim=32), UNSUPPORTED),
    (dict(head_dim=272, rot_dim=32, q_stride=1 << 20, k_stride=1 << 20, q_out_stride=1 << 20), UNSUPPORTED),
    (dict(num_heads=0), INVALID), (dict(num_tokens=-1), INVALID), (dict(num_tokens=0, q=None, k_out=None), pa.PA_OK),
])
def test_norm_rope_refusals(lib, kw, status):
    assert _norm(lib, **kw) == status


def test_packed_arguments_are_the_header_s_struct():
    import struct
    assert struct.calcsize("@PPqqPqPPffPPP10i") == ctypes.sizeof(pa._NormRopeArgs)
    values = list(range(1, 9)) + [0.5, 0.25] + list(range(9, 12)) + list(range(20, 30))
    s = pa._NormRopeArgs.from_buffer_copy(pa._norm_rope_pack(*values))
    got = [getattr(s, n) for n, _ in s._fields_ if n != "pair_axis"]
    assert got == values[:12] + values[13:]


def test_norm_rope_append_refusals(lib):
    def pool(v=FAKE, v_stride=256, slots=FAKE, kc=FAKE, vc=FAKE, bs=16, nb=4, **kw):
        args = pa._NormRopeArgs(**{**NORM, **kw})
        return lib.pa_norm_rope_append(ctypes.byref(args), v, v_stride, slots, kc, vc, bs, nb, None, None)

    def pool4(kp=FAKE, vp=FAKE, slots=FAKE, **kw):
        args = pa._NormRopeArgs(**{**NORM, **kw})
        return lib.pa_norm_rope_append_int4(ctypes.byref(args), FAKE, 256, slots, FAKE, FAKE, kp, vp, 16, 4, None, None)

    for kw in (dict(v=None), dict(v=FAKE + 8), dict(v_stride=100), dict(v_stride=260), dict(slots=None),
               dict(slots=FAKE + 4), dict(kc=None), dict(vc=FAKE + 8), dict(bs=0), dict(nb=0)):
        assert pool(**kw) == INVALID, kw
    assert pool4(kp=None) == INVALID and pool4(vp=FAKE + 4) == INVALID and pool4(slots=None) == INVALID
    assert pool4(head_dim=48, rot_dim=48) == UNSUPPORTED
    assert pool(num_tokens=0) == pa.PA_OK and pool4(num_tokens=0) == pa.PA_OK
    assert lib.pa_norm_rope(None, FAKE, 256, None, None) == INVALID


def test_int4_pools_copy_by_their_byte_rows(lib):
    """pa_copy_blocks takes PA_DTYPE_INT4 with the number of dims."""
    def copy(d):
        return lib.pa_copy_blocks(None, None, None, 1, 2, d, 16, 8, 4, None, None)
    assert copy(48) == UNSUPPORTED and copy(33) == UNSUPPORTED and copy(64) == INVALID   # null pools
    assert pa.pa_default_partition_size("int4") == 1024


# ------------------------------------------------------------------ binding


@dataclasses.dataclass
class _Shapes:
    B: int = 2
    hq: int = 8
    hkv: int = 2
    d: int = 128
    nb: int = 8
    bs: int = 16


def _dev(shape, dtype=torch.bfloat16, index=0):
    t = _OnDevice(shape, dtype, index)
    t.stride = lambda *a: t._t.stride(*a)
    return t


def _pool(z, index=0):
    return [_dev((z.nb, z.hkv, z.bs, z.d // 2), torch.uint8, index) for _ in range(2)] + \
        [_dev((z.nb, z.hkv, z.bs, 2), torch.bfloat16, index) for _ in range(2)]


@pytest.fixture
def no_library(monkeypatch):
    def reached():
        raise AssertionError("the library was reached")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(pa, "lib", reached)


def test_binding_refuses_other_devices_and_shapes(no_library):
    z = _Shapes()
    q, out = _dev((z.B, z.hq, z.d)), _dev((z.B, z.hq, z.d))
    bt, cl, ws = _dev((z.B, 4), torch.int32), _dev((z.B,), torch.int32), _dev((4096,), torch.uint8)
    slots, rows = _dev((z.B,), torch.int64), _dev((z.B, z.hkv, z.d))

    def decode(q=q, pool=None, bt=bt, out=out, ws=ws):
        pa.pa_decode_int4(q, *(pool or _pool(z)), bt, cl, 0.1, out, 64, workspace=ws)

    with pytest.raises(AssertionError, match="reached"):
        decode()
    for kw in (dict(q=_dev((z.B, z.hq, z.d), index=1)), dict(pool=_pool(z, 1)), dict(ws=_dev((9,), torch.uint8, 1))):
        with pytest.raises(ValueError, match="current CUDA device"):
            decode(**kw)
    for kw in (dict(bt=_dev((3, 4), torch.int32)), dict(out=_dev((z.B, 1, z.hq, z.d))), dict(q=_dev((z.B, z.hq, 64)))):
        with pytest.raises(ValueError, match="mismatch"):
            decode(**kw)
    with pytest.raises(TypeError):
        decode(q=_dev((z.B, z.hq, z.d), torch.float32))
    p = _pool(z)
    with pytest.raises(ValueError, match="INT4 pools"):
        pa.pa_reshape_and_cache_int4(rows, rows, slots, p[0], p[1], p[2], _dev((z.nb, z.hkv, z.bs, 1)))
    with pytest.raises(ValueError, match="mismatch"):
        pa.pa_reshape_and_cache_int4(rows, rows, _dev((3,), torch.int64), *p)
    with pytest.raises(ValueError, match="mismatch"):
        pa.pa_gather_int4(*p, bt, cl, slots, rows, _dev((3, z.hkv, z.d)), 64)
    with pytest.raises(AssertionError, match="reached"):
        pa.pa_gather_int4(*p, bt, cl, slots, rows, rows, 64)


def test_norm_rope_binding_checks(no_library):
    z = _Shapes()
    q, k = _dev((z.B, z.hq, z.d)), _dev((z.B, z.hkv, z.d))
    pos, table = _dev((z.B,), torch.int32), _dev((50, 64), torch.float32)

    def call(q=q, k=k, pos=pos, table=table, q_out=None, k_out=None, **kw):
        pa.pa_norm_rope(q, k, pos, table, q_out or q, k_out or k, **kw)

    with pytest.raises(AssertionError, match="reached"):
        call(q_weight=_dev((z.d,)), pair_axis=[0] * 32)
    for kw, what in [(dict(pos=_dev((3,), torch.int32)), "positions"), (dict(pair_axis=[0] * 31), "pair_axis"),
                     (dict(table=None), "need cos_sin"), (dict(q_weight=_dev((64,))), "head_dim"),
                     (dict(k_out=_dev((z.B, 3, z.d))), "mismatch"), (dict(k=_dev((3, z.hkv, z.d))), "mismatch"),
                     (dict(k_weight=_dev((z.d,), index=1)), "current CUDA device")]:
        with pytest.raises(ValueError, match=what):
            call(**kw)
    with pytest.raises(TypeError):
        call(q_weight=_dev((z.d,)), k_weight=_dev((z.d,), torch.float32))
    bent = _dev((z.B, z.hq, z.d))
    bent.stride = lambda *a: (z.hq * z.d, z.d + 8, 1)
    with pytest.raises(ValueError, match="contiguous"):
        call(q=bent)
    cpu = torch.zeros(z.B, z.hq, z.d, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        call(q=cpu)
    slots = _dev((z.B,), torch.int64)
    pool = [_dev((z.nb, z.hkv, z.bs, z.d)) for _ in range(2)]
    with pytest.raises(AssertionError, match="reached"):
        pa.pa_norm_rope_append(q, k, k, pos, table, slots, q, *pool)
    with pytest.raises(TypeError):
        f32 = [_dev((z.nb, z.hkv, z.bs, z.d), torch.float32) for _ in range(2)]
        pa.pa_norm_rope_append(q, k, k, pos, table, slots, q, *f32)
    with pytest.raises(ValueError, match="mismatch"):
        pa.pa_norm_rope_append(q, k, k, pos, table, _dev((3,), torch.int64), q, *pool)
    with pytest.raises(AssertionError, match="reached"):
        pa.pa_norm_rope_append_int4(q, k, k, pos, table, slots, q, *_pool(z))
