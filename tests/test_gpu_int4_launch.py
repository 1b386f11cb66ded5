"""Launch sizes of the 4-bit append and gather: bounds far above the lengths, and
tokens whose heads several warps share."""
import numpy as np
import pytest
import torch

import rows_reference as ref
from paged_kv_cache_29_gb300 import _binding as pa
from test_gpu_int4 import Batch, bf16, dev, host

pytestmark = pytest.mark.gpu


def _timed(call):
    call()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    call()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b)


def test_gather_with_the_largest_length_bound():
    """max_context_len up to 2^31 - 1 says nothing about the lengths: the rows are the
    same, and as many CTAs share them (one CTA would take over 50 times as long)."""
    b = Batch([60_000], hq=1, hkv=1, d=64, bs=256, seed=41).upload()
    width = (1 << 31) // 256
    table = torch.zeros(1, width, dtype=torch.int32, device="cuda")
    table[:, :b.table.shape[1] - 1] = b.dtable[:, :-1]
    k = torch.empty(60_000, 1, 64, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    start = torch.zeros(1, dtype=torch.int64, device="cuda")

    def gather(t, bound):
        pa.pa_gather_int4(*b.dpools, t, b.dlens, start, k, v, bound, error_word=b.err)

    near = _timed(lambda: gather(b.dtable, b.mcl))
    want = k.clone(), v.clone()
    k.zero_(), v.zero_()
    far = _timed(lambda: gather(table, 2 ** 31 - 1))
    assert int(b.err.item()) == 0
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
    i = np.arange(60_000)
    for got, c, p in ((k, 0, 2), (v, 1, 3)):
        x = ref.values4(b.pools[c][b.table[0, i // 256], :, i % 256], b.pools[p][b.table[0, i // 256], :, i % 256])
        np.testing.assert_array_equal(host(got), ref.bf16_of_double(x))
    assert far < 8 * near, (near, far)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,hkv", [(1, 32), (3, 130), (300, 32), (700, 32), (1400, 32), (1500, 32), (2800, 32)])
def test_tokens_whose_heads_several_warps_share(T, hkv, dtype):
    rng = np.random.default_rng(T)
    x = rng.standard_normal((2, T, hkv, 128)).astype(np.float32)
    if dtype == "bf16":
        bits = bf16(x)
        x, dx = ref.bf16_value(bits), [dev(b) for b in bits]
    else:
        dx = [dev(a) for a in x]
    nb = T // 16 + 2
    pools = [torch.full((nb, hkv, 16, 64), 9, dtype=torch.uint8, device="cuda") for _ in range(2)] + \
        [torch.full((nb, hkv, 16, 2), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    slots = rng.permutation(nb * 16)[:T].astype(np.int64)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_reshape_and_cache_int4(*dx, dev(slots), *pools, error_word=err)
    assert int(err.item()) == 0
    free = np.setdiff1d(np.arange(nb * 16), slots)
    for rows, c, p in ((x[0], 0, 2), (x[1], 1, 3)):
        codes, pairs = ref.quantise4(rows)
        got_codes, got_pairs = host(pools[c]), host(pools[p])
        np.testing.assert_array_equal(got_codes[slots // 16, :, slots % 16], codes)
        np.testing.assert_array_equal(got_pairs[slots // 16, :, slots % 16], pairs)
        assert (got_codes[free // 16, :, free % 16] == 9).all()
