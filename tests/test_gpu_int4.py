"""The 4-bit cache on the GPU: append and gather bit for bit, decode attention
within a derived bound of a 64-bit reference on the same codes and pairs
(rows_reference.attention4 says what the bound counts)."""
import numpy as np
import pytest
import torch

import rows_reference as ref
from paged_kv_cache_29_gb300 import _binding as pa

pytestmark = pytest.mark.gpu


def dev(a):
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int16)).view(torch.bfloat16).cuda() if a.dtype == np.uint16 else torch.from_numpy(a).cuda()


def host(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16) if t.dtype == torch.bfloat16 else t.cpu().numpy()


def bf16(x):
    return ref.bf16_bits(np.asarray(x, np.float32))


def value(bits):
    return ref.bf16_value(bits).astype(np.float64)


class Batch:
    """A pool of quantised rows, block tables in random order (entries past a
    sequence's end are garbage) and q."""

    def __init__(self, lens, hq=8, hkv=2, d=128, bs=16, Q=1, seed=0, k_gain=1.0, v_gain=1.0, spare=2, v_shift=0.0):
        rng = np.random.default_rng(seed)
        self.lens, self.hq, self.hkv, self.d, self.bs, self.Q = lens, hq, hkv, d, bs, Q
        nblk = [-(-n // bs) for n in lens]
        self.nb = sum(nblk) + spare
        perm = rng.permutation(self.nb)
        width = max(1, max(nblk, default=0)) + 1
        self.table = np.where(rng.random((len(lens), width)) < 0.5, -7, 1 << 30).astype(np.int32)
        at = 0
        for s, m in enumerate(nblk):
            self.table[s, :m] = perm[at:at + m]
            at += m
        shape = (self.nb, hkv, bs, d)
        k = (rng.standard_normal(shape) * k_gain).astype(np.float32)
        k[..., ::9] *= 2
        v = (rng.standard_normal(shape) * v_gain + v_shift).astype(np.float32)
        (kc, kp), (vc, vp) = ref.quantise4(k), ref.quantise4(v)
        self.pools = [kc, vc, kp, vp]
        self.q = bf16(rng.standard_normal((len(lens), Q, hq, d)))
        self.scale = d ** -0.5 / k_gain
        self.mcl = max(list(lens) + [0])

    def upload(self):
        self.dq = dev(self.q if self.Q > 1 else self.q[:, 0])
        self.dpools = [dev(p) for p in self.pools]
        self.dtable, self.dlens = dev(self.table), dev(np.array(self.lens, np.int32))
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.out = torch.full_like(self.dq, float("nan"))
        return self

    def decode(self, window=0, **kw):
        pa.pa_decode_int4(self.dq, *self.dpools, self.dtable, self.dlens, self.scale, self.out, kw.pop("mcl", self.mcl),
                          window=window, error_word=self.err, **kw)
        torch.cuda.synchronize()
        return value(host(self.out)).reshape(len(self.lens), self.Q, self.hq, self.d)

    def check(self, got, window=0, skip=()):
        for s, n in enumerate(self.lens):
            if s in skip:
                continue
            want, tol = ref.attention4(value(self.q[s]), self.pools, self.table[s], n, self.scale, self.bs, window)
            worst = np.max(np.abs(got[s] - want) - tol)
            assert worst <= 0, f"sequence {s} of {n} rows: {worst:.3g} over its bound"


RAGGED = [1, 15, 16, 0, 17, 100, 511, 512, 513, 1030, 3000, 2]
EDGES = [1023, 1024, 1025, 1040, 1151, 1152, 1153, 2047, 2048, 2175, 2176, 2177, 3200, 3201]   # of partitions and their tails


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 6, 7, 8])
def test_decode_ragged_groups(group, d):
    b = Batch(RAGGED, hq=3 * group, hkv=3, d=d, seed=group + d).upload()
    got = b.decode()
    assert int(b.err.item()) == 0
    b.check(got)


@pytest.mark.parametrize("d,hq,Q", [(64, 4, 1), (128, 4, 1), (128, 4, 2)])
def test_decode_partition_edges(d, hq, Q):
    b = Batch(EDGES, hq=hq, hkv=1, d=d, Q=Q, seed=d).upload()
    b.check(b.decode())
    b.check(b.decode(1024), 1024)
    assert int(b.err.item()) == 0


@pytest.mark.parametrize("bs", [32, 48, 256])
def test_decode_block_sizes(bs):
    b = Batch(RAGGED, hq=8, hkv=2, bs=bs, seed=bs).upload()
    b.check(b.decode())
    assert int(b.err.item()) == 0


@pytest.mark.parametrize("window", [1, 5, 16, 17, 100, 512, 530, 2999, 3000, 2 ** 31 - 1])
def test_decode_windows(window):
    b = Batch(RAGGED, hq=8, hkv=2, seed=3).upload()
    b.check(b.decode(window), window)
    assert int(b.err.item()) == 0


@pytest.mark.parametrize("group,Q", [(1, 8), (2, 4), (4, 2), (2, 3), (1, 5)])
@pytest.mark.parametrize("window", [0, 1, 40, 700])
def test_decode_several_queries(group, Q, window):
    lens = [Q, Q + 1, 16, 17, 0, 33, 512, 513, 514, 1030, 2050]
    b = Batch(lens, hq=2 * group, hkv=2, Q=Q, seed=Q).upload()
    b.check(b.decode(window), window)
    assert int(b.err.item()) == 0


@pytest.mark.parametrize("k_gain,v_gain,v_shift", [(1e4, 1e-6, 0.0), (1e-6, 1e6, 0.0), (1.0, 1e-30, 0.0), (1e15, 1e20, 0.0),
                                                   (1.0, 0.01, 30.0)])
def test_decode_magnitudes(k_gain, v_gain, v_shift):
    b = Batch([3, 70, 600, 1100], hq=8, hkv=2, seed=5, k_gain=k_gain, v_gain=v_gain, v_shift=v_shift).upload()
    b.check(b.decode())


def test_decode_mixed_value_scales_and_constant_rows():
    """V rows whose steps span 2^60, among them rows of one value (step 0)."""
    b = Batch([40, 300, 700], hq=8, hkv=2, seed=6)
    rng = np.random.default_rng(7)
    v = rng.standard_normal((b.nb, b.hkv, b.bs, b.d)) * 2.0 ** rng.integers(-40, 20, (b.nb, b.hkv, b.bs, 1))
    v[rng.random((b.nb, b.hkv, b.bs)) < 0.2] = 0.75
    b.pools[1], b.pools[3] = ref.quantise4(v.astype(np.float32))
    b.upload()
    b.check(b.decode())


def test_decode_only_constant_rows():
    b = Batch([1, 17, 600], hq=4, hkv=2, seed=8)
    b.pools[1], b.pools[3] = ref.quantise4(np.full((b.nb, b.hkv, b.bs, b.d), -3.0, np.float32))
    got = b.upload().decode()
    assert (got == -3.0).all()


def test_decode_small_and_large_queries():
    for gain in (2.0 ** -40, 2.0 ** 60, 0.0):
        b = Batch([5, 600], hq=8, hkv=2, seed=9)
        b.q = bf16(value(b.q) * gain)
        b.scale = b.scale / gain if gain else b.scale
        b.upload()
        b.check(b.decode())


def test_decode_peaked_softmax():
    """Scores far apart (one row takes all the weight, at either end and in between)."""
    b = Batch([700, 33, 513], hq=8, hkv=2, seed=10)
    b.scale *= 60
    b.upload()
    b.check(b.decode())


@pytest.mark.parametrize("factor", [-1.0, 0.0, -40.0])
def test_negative_and_zero_scales(factor):
    b = Batch([5, 600, 1500], hq=8, hkv=2, seed=25)
    b.scale *= factor
    b.upload()
    b.check(b.decode())


def test_infinite_and_nan_queries_stay_in_their_rows():
    b = Batch([40, 700, 1300], hq=8, hkv=2, seed=26)
    clean = b.q.copy()
    b.q[0, 0, 1, 5], b.q[1, 0, 4, 0], b.q[2, 0, 7, 127] = 0x7FC0, 0x7F80, 0xFF80      # NaN, inf, -inf
    got = b.upload().decode()
    b.q = clean
    for s, h in ((0, 1), (1, 4), (2, 7)):
        assert not np.isfinite(got[s, 0, h]).all()
        want, _ = ref.attention4(value(b.q[s]), b.pools, b.table[s], b.lens[s], b.scale, b.bs)
        got[s, 0, h] = want[0, h]
    b.check(got)


def test_a_sequence_with_a_nan_row_leaves_the_others_alone():
    b = Batch([600, 40, 1100], hq=8, hkv=2, seed=27)
    for pairs in b.pools[2:]:
        pairs[b.table[0, 3], 1, 5] = [0x7FC0, 0x7F80]
    got = b.upload().decode()
    assert np.isnan(got[0, 0, 4:]).all()                            # the heads of KV head 1
    b.check(got, skip=(0,))


def test_garbage_past_the_end_does_not_leak():
    lens = [1, 17, 40, 600]
    b = Batch(lens, hq=8, hkv=2, seed=11)
    for s, n in enumerate(lens):
        for i in range(n, -(-n // b.bs) * b.bs):
            for pairs in b.pools[2:]:
                pairs[b.table[s, i // b.bs], :, i % b.bs] = [0x7FC0, 0x7F80]    # NaN, inf
    b.upload()
    with np.errstate(invalid="ignore"):
        b.check(b.decode())
    b2 = Batch(lens, hq=8, hkv=2, seed=11)
    for s, n in enumerate(lens):                                    # rows before a window
        for i in range(max(0, n - 7)):
            for pairs in b2.pools[2:]:
                pairs[b2.table[s, i // b2.bs], :, i % b2.bs] = [0x7FC0, 0xFF80]
    b2.upload()
    b2.check(b2.decode(7), 7)


def test_flagged_sequences_leave_the_others_alone():
    b = Batch([600, 40, 3, 700, 90], hq=8, hkv=2, Q=2, seed=12)
    b.lens[2] = 1                                                   # fewer rows than query tokens
    b.table[3, 2] = b.nb                                            # outside the pool
    b.upload()
    b.dlens[0] = -4
    b.dlens[1] = 10 ** 6
    got = b.decode(mcl=720)
    assert int(b.err.item()) == pa.PA_DEVERR_CONTEXT | pa.PA_DEVERR_BLOCK_ID
    assert np.isnan(got[:3]).all()                                  # left as they were
    b.check(got, skip=(0, 1, 2, 3))


@pytest.mark.parametrize("hq,lens,Q", [(1, [2100], 1), (3, [2100], 1), (1, [1025, 3000, 40], 3), (5, [1100, 2049, 7], 1)])
def test_odd_numbers_of_partials(hq, lens, Q):
    """Partials whose maxima and sums end off a 16-byte boundary."""
    b = Batch(lens, hq=hq, hkv=1, d=128, Q=Q, seed=hq).upload()
    b.check(b.decode())
    assert int(b.err.item()) == 0


def test_batch_invariance_is_bitwise():
    lens = [700, 33, 4000, 1, 515, 0, 2047]
    b = Batch(lens, hq=8, hkv=2, seed=13).upload()
    b.decode()
    whole = b.out.clone()
    for s in range(len(lens)):
        out = torch.full_like(whole[s:s + 1], float("nan"))
        pa.pa_decode_int4(b.dq[s:s + 1], *b.dpools, b.dtable[s:s + 1], b.dlens[s:s + 1], b.scale, out, b.mcl)
        assert torch.equal(out.view(torch.int16), whole[s:s + 1].view(torch.int16)), s
    again = torch.full_like(whole, float("nan"))
    pa.pa_decode_int4(b.dq, *b.dpools, b.dtable, b.dlens, b.scale, again, b.mcl)
    assert torch.equal(again.view(torch.int16), whole.view(torch.int16))


def test_long_sequence_beside_short_ones():
    b = Batch([40_000, 20, 1500, 3], hq=4, hkv=1, seed=14).upload()
    b.check(b.decode())


def test_merges_of_many_partitions():
    """One warp's 16 partitions, one more, and more than 16 warps take at once."""
    b = Batch([128 + 16 * 1024, 129 + 16 * 1024, 300_000], hq=1, hkv=1, d=64, seed=15).upload()
    b.check(b.decode())


def test_more_sequences_than_one_launch_holds():
    rng = np.random.default_rng(15)
    b = Batch([int(n) for n in rng.integers(0, 40, 4400)], hq=2, hkv=1, d=64, seed=16).upload()
    b.check(b.decode())
    assert int(b.err.item()) == 0


def test_more_items_than_a_cta_keeps_in_shared_memory():
    rng = np.random.default_rng(28)
    lens = [int(n) for n in rng.integers(0, 36, 3000)]
    b = Batch(lens, hq=8, hkv=8, d=64, seed=29).upload()            # some 50 items for each of 456 CTAs
    b.check(b.decode(), skip=set(range(3000)) - set(rng.permutation(3000)[:400].tolist()))
    assert int(b.err.item()) == 0


def test_empty_batch_and_empty_sequences():
    b = Batch([0, 0], hq=8, hkv=2, seed=17).upload()
    assert (b.decode() == 0).all()
    pa.pa_decode_int4(b.dq[:0], *b.dpools, b.dtable[:0], b.dlens[:0], b.scale, b.out[:0], 0)


def test_graphs_share_a_workspace_and_follow_their_inputs():
    """Two captured calls on one workspace, replayed in turn on new inputs."""
    b1 = Batch([600, 33, 1200], hq=8, hkv=2, seed=18).upload()
    b2 = Batch([90, 2000], hq=8, hkv=2, seed=19).upload()
    ws = torch.empty(max(pa.pa_decode_workspace_size_multi(len(b.lens), 1, 8, 128, b.mcl) for b in (b1, b2)), dtype=torch.uint8,
                     device="cuda")
    b1.decode(workspace=ws), b2.decode(workspace=ws)
    graphs = []
    side = torch.cuda.Stream()
    for b in (b1, b2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            pa.pa_decode_int4(b.dq, *b.dpools, b.dtable, b.dlens, b.scale, b.out, b.mcl, workspace=ws, error_word=b.err)
        graphs.append(g)
    for seed in (20, 21):
        for b in (b1, b2):
            b.q = bf16(np.random.default_rng(seed + len(b.lens)).standard_normal(b.q.shape))
            b.dq.copy_(dev(b.q[:, 0]))
            b.out.fill_(float("nan"))
        b1.lens[0] = 600 - seed
        b1.dlens[0] = 600 - seed
        for _ in range(2):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        for b in (b1, b2):
            b.check(value(host(b.out))[:, None])


def test_two_streams_with_their_own_workspaces():
    b1 = Batch([1600, 33, 1200] * 8, hq=8, hkv=2, seed=22).upload()
    b2 = Batch([90, 2000] * 8, hq=8, hkv=2, seed=23).upload()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    ws = [torch.empty(pa.pa_decode_workspace_size_multi(len(b.lens), 1, 8, 128, b.mcl), dtype=torch.uint8, device="cuda")
          for b in (b1, b2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for b, st, w in zip((b1, b2), streams, ws):
            pa.pa_decode_int4(b.dq, *b.dpools, b.dtable, b.dlens, b.scale, b.out, b.mcl, workspace=w, error_word=b.err, stream=st)
    torch.cuda.synchronize()
    for b in (b1, b2):
        b.check(value(host(b.out))[:, None])


def test_offsets_past_32_bits():
    """A pool of more than 4 GiB of codes, its last blocks in use."""
    small = Batch([40, 700], hq=8, hkv=8, seed=24)
    nb = (1 << 32) // (8 * 16 * 64) + 4096
    used = small.nb
    pools = []
    for p in small.pools:
        big = torch.empty((nb,) + p.shape[1:], dtype=torch.uint8 if p.dtype == np.uint8 else torch.bfloat16, device="cuda")
        big[nb - used:] = dev(p)
        pools.append(big)
    small.upload()
    table = torch.where((small.dtable >= 0) & (small.dtable < used), small.dtable + (nb - used), small.dtable)
    pa.pa_decode_int4(small.dq, *pools, table, small.dlens, small.scale, small.out, small.mcl, error_word=small.err)
    small.check(value(host(small.out))[:, None])
    k = torch.empty(740, 8, 128, dtype=torch.float32, device="cuda")
    v = torch.empty_like(k)
    starts = torch.tensor([0, 40], device="cuda")
    pa.pa_gather_int4(*pools, table, small.dlens, starts, k, v, small.mcl, error_word=small.err)
    row = torch.randn(1, 8, 128, device="cuda").bfloat16()
    slot = torch.tensor([nb * 16 - 1], device="cuda")
    pa.pa_reshape_and_cache_int4(row, row, slot, *pools, error_word=small.err)
    torch.cuda.synchronize()
    assert int(small.err.item()) == 0
    i = np.arange(40)
    want = ref.values4(small.pools[0][small.table[0, i // 16], :, i % 16], small.pools[2][small.table[0, i // 16], :, i % 16])
    np.testing.assert_array_equal(k[:40].cpu().numpy(), want.astype(np.float32))
    codes, pairs = ref.quantise4(row.float().cpu().numpy())
    np.testing.assert_array_equal(pools[0][-1, :, -1].cpu().numpy(), codes[0])
    np.testing.assert_array_equal(host(pools[2][-1, :, -1]), pairs[0])


# ----------------------------------------------------------- append, gather


def _rows(rng, T, hkv, d, dtype):
    x = rng.standard_normal((T, hkv, d)) * 10.0 ** rng.uniform(-4, 4, (T, hkv, 1)) + rng.uniform(-2, 2, (T, hkv, 1))
    x[T // 2] = 0.0
    x[T // 3] = 1.25
    x[T // 4] = np.where(rng.random((hkv, d)) < 0.5, 0.0, -0.0)
    x[T // 5] *= 1e-33                       # steps too small for the shared reciprocal
    x[T // 6] *= 1e30
    x = x.astype(np.float32)
    if dtype == "f32":
        return x, dev(x)
    b = bf16(x)
    return ref.bf16_value(b), dev(b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 96, 128, 160, 256])
@pytest.mark.parametrize("bs", [1, 7, 16])
def test_append_and_gather_are_bit_exact(dtype, d, bs):
    rng = np.random.default_rng(d + bs)
    hkv, T = 3, 61
    nb = 90 // bs + 3
    k, dk = _rows(rng, T, hkv, d, dtype)
    v, dv = _rows(rng, T, hkv, d, dtype)
    pools = [rng.integers(0, 256, (nb, hkv, bs, d // 2)).astype(np.uint8) for _ in range(2)] + \
        [bf16(rng.standard_normal((nb, hkv, bs, 2))) for _ in range(2)]
    slots = rng.permutation(nb * bs)[:T].astype(np.int64)
    slots[3], slots[9], slots[10] = -1, nb * bs, 1 << 40
    dp = [dev(p) for p in pools]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_reshape_and_cache_int4(dk, dv, dev(slots), *dp, error_word=err)
    assert int(err.item()) == pa.PA_DEVERR_SLOT
    for t, s in enumerate(slots):
        if 0 <= s < nb * bs:
            for x, c, p in ((k, 0, 2), (v, 1, 3)):
                pools[c][s // bs, :, s % bs], pools[p][s // bs, :, s % bs] = ref.quantise4(x[t])
    for got, want in zip(dp, pools):
        np.testing.assert_array_equal(host(got), want)

    # Everything back through tables, in both types, between rows left alone.
    lens = [0, 1, bs, 2 * bs + 1, 5]
    width = 4 + 5 // bs
    table = rng.integers(0, nb, (5, width)).astype(np.int32)
    starts = np.array([2, 3, 5, 24, 60], np.int64)
    for out_dtype in (torch.bfloat16, torch.float32):
        out = [torch.full((70, hkv, d), 7.0, dtype=out_dtype, device="cuda") for _ in range(2)]
        pa.pa_gather_int4(*dp, dev(table), dev(np.array(lens, np.int32)), dev(starts), *out, width * bs, error_word=err)
        for o, c, p in ((out[0], 0, 2), (out[1], 1, 3)):
            want = np.full((70, hkv, d), 7.0, np.float32)
            for s, n in enumerate(lens):
                i = np.arange(n)
                blk = table[s, i // bs]
                want[starts[s] + i] = ref.values4(pools[c][blk, :, i % bs], pools[p][blk, :, i % bs]).astype(np.float32)
            got = host(o)
            np.testing.assert_array_equal(got, bf16(want) if out_dtype == torch.bfloat16 else want)


def test_gather_flags_and_skips():
    b = Batch([40, 33, 20, 17, 10], hq=2, hkv=2, d=64, seed=30)
    b.table[1, 1] = b.nb                                         # one bad block
    b.upload()
    b.dlens[2] = 1000
    starts = np.array([0, 40, 73, 190, -1], np.int64)            # the fourth passes the end, the last is before the start
    k = torch.full((200, 2, 64), 7.0, device="cuda")
    v = k.clone()
    pa.pa_gather_int4(*b.dpools, b.dtable, b.dlens, dev(starts), k, v, 48, error_word=b.err)
    assert int(b.err.item()) == pa.PA_DEVERR_CONTEXT | pa.PA_DEVERR_BLOCK_ID
    i = np.arange(40)
    want = ref.values4(b.pools[1][b.table[0, i // 16], :, i % 16], b.pools[3][b.table[0, i // 16], :, i % 16])
    got = v.cpu().numpy()
    np.testing.assert_array_equal(got[:40], want.astype(np.float32))
    assert (got[56:72] == 7.0).all()                             # the bad block's rows
    assert (got[73:] == 7.0).all()                               # the flagged sequences'
    pa.pa_gather_int4(*b.dpools, b.dtable[:0], b.dlens[:0], dev(starts[:0]), k, v, 48)


def test_large_append_and_gather():
    """More rows than one grid's threads, one long sequence beside short ones."""
    rng = np.random.default_rng(31)
    lens = [9000, 3, 0, 700]
    b = Batch(lens, hq=8, hkv=8, d=128, seed=32).upload()
    total = sum(lens)
    seq = np.repeat(np.arange(4), lens)
    row = np.concatenate([np.arange(n) for n in lens])
    slots = b.table[seq, row // 16].astype(np.int64) * 16 + row % 16
    x = bf16(rng.standard_normal((2, total, 8, 128)))
    pa.pa_reshape_and_cache_int4(dev(x[0]), dev(x[1]), dev(slots), *b.dpools, error_word=b.err)
    k = torch.empty(total, 8, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    starts = np.concatenate([[0], np.cumsum(lens)[:-1]]).astype(np.int64)
    pa.pa_gather_int4(*b.dpools, b.dtable, b.dlens, dev(starts), k, v, b.mcl, error_word=b.err)
    assert int(b.err.item()) == 0
    for i, got in enumerate((k, v)):
        want = ref.values4(*ref.quantise4(ref.bf16_value(x[i])))
        np.testing.assert_array_equal(host(got), ref.bf16_of_double(want))


def test_copy_on_write_of_a_4_bit_pool():
    b = Batch([40, 600, 17], hq=8, hkv=2, seed=33, spare=8).upload()
    used = {int(x) for s, n in enumerate(b.lens) for x in b.table[s, :-(-n // 16)]}
    free = [x for x in range(b.nb) if x not in used][:6]
    pairs = dev(np.array(list(zip(sorted(used), free)), np.int64))
    kc, vc, kp, vp = b.dpools
    pa.pa_copy_blocks(kc, vc, pairs, error_word=b.err)
    pa.pa_copy_blocks(kp.view(b.nb, 1, 1, -1), vp.view(b.nb, 1, 1, -1), pairs, error_word=b.err)
    assert int(b.err.item()) == 0
    for src, dst in pairs.tolist():
        for got, p in zip(b.dpools, b.pools):
            np.testing.assert_array_equal(host(got[dst]), p[src])
    # the C call takes the dims and PA_DTYPE_INT4
    rc = pa.lib().pa_copy_blocks(kc.data_ptr(), vc.data_ptr(), pairs.data_ptr(), len(free), 2, 128, 16, b.nb, 4,
                                 b.err.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert rc == pa.PA_OK
    torch.cuda.synchronize()
