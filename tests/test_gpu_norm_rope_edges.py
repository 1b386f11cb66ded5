"""Norm and rotation calls at the edges of their values: dims past rot_dim and
rows without a norm pass through, whatever stands beside them."""
import numpy as np
import pytest
import torch

from paged_kv_cache_29_gb300 import _binding as pa
from test_gpu_int4 import dev, host
from test_gpu_norm_rope import Rows

pytestmark = pytest.mark.gpu


def _any_values(rng, shape, dtype):
    """Every kind of value but NaN: infinities, zeros of both signs, subnormals."""
    if dtype == "bf16":
        bits = rng.integers(0, 1 << 16, shape).astype(np.uint16)
        special = np.array([0x7F80, 0xFF80, 0x0000, 0x8000, 0x0001, 0x8001], np.uint16)
        nan = (bits & 0x7FFF) > 0x7F80
    else:
        bits = rng.integers(0, 1 << 32, shape, dtype=np.uint64).astype(np.uint32)
        special = np.array([0x7F800000, 0xFF800000, 0, 0x80000000, 1, 0x80000001], np.uint32)
        nan = (bits & 0x7FFFFFFF) > 0x7F800000
    return np.where(nan | (rng.random(shape) < 0.4), rng.choice(special, shape), bits)


def _upload(bits):
    return dev(bits if bits.dtype == np.uint16 else bits.view(np.float32))


def _bits(t):
    return host(t) if t.dtype == torch.bfloat16 else t.cpu().numpy().view(np.uint32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,rot", [(64, 0), (128, 0), (128, 32), (96, 48), (256, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_dims_that_are_not_turned_pass_through(dtype, d, rot, interleaved):
    """Without norms, dims past rot_dim arrive bit for bit: an infinity stays in
    its own dim, a zero keeps its sign; the turned dims are what they are
    beside ordinary values."""
    T, hq, hkv, bs, nb = 9, 3, 2, 4, 4
    rng = np.random.default_rng(d + rot)
    r = Rows(T, hq, hkv, d, dtype, rot, seed=d + rot + 1)
    q, k, v = (t.contiguous() for t in r.parts(r.dqkv))
    qb, kb = _bits(q).copy(), _bits(k).copy()
    qb[..., rot:] = _any_values(rng, qb[..., rot:].shape, dtype)
    kb[..., rot:] = _any_values(rng, kb[..., rot:].shape, dtype)
    q, k = _upload(qb), _upload(kb)
    pos, cs = r.position_args()
    q_out, k_out = r.out(hq), r.out(hkv)
    pa.pa_norm_rope(q, k, pos, cs, q_out, k_out, interleaved=interleaved)
    kc = torch.zeros(nb, hkv, bs, d, dtype=q.dtype, device="cuda")
    q_two = r.out(hq)
    pa.pa_norm_rope_append(q, k, v, pos, cs, dev(np.arange(T, dtype=np.int64)), q_two, kc, torch.zeros_like(kc), interleaved=interleaved)
    pool = kc.transpose(1, 2).reshape(nb * bs, hkv, d)[:T]
    for got, bits in ((q_out, qb), (q_two, qb), (k_out, kb), (pool, kb)):
        np.testing.assert_array_equal(_bits(got)[..., rot:], bits[..., rot:])
    if rot:
        for which, got in ((0, q_out), (1, k_out)):
            want, size = r.want(which, weight=None, interleaved=interleaved)
            half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
            off = np.abs(r.read(got) - want)[..., :rot]
            assert (off <= (half * np.abs(want) + 2.0 ** -20 * size)[..., :rot]).all()


def test_nan_past_the_rotation_stays_in_its_dim():
    r = Rows(4, 2, 2, 128, rot=64, seed=5)
    q, k, _ = (t.contiguous() for t in r.parts(r.dqkv))
    clean = q.clone()
    q[:, :, 64::2] = float("nan")
    q_out = r.out(2)
    pa.pa_norm_rope(q, k, *r.position_args(), q_out, r.out(2))
    assert torch.isnan(q_out[..., 64::2]).all()
    assert torch.equal(q_out[..., 65::2], clean[..., 65::2])
