"""pa_decode_sinks and pa_decode_weights against 64 bits."""
import numpy as np
import pytest
import torch

import cache_rows_reference as ref
import paged_kv_cache_29_gb300 as pkg
from paged_kv_cache_29_gb300 import _binding as pa

pytestmark = pytest.mark.gpu

# (dtype, query heads per KV head, tokens, head_dim, block_size): shapes of the tile
# ring, then shapes that it has no instance for.
RING = [("bf16", 1, 1, 128, 16), ("bf16", 4, 1, 128, 16), ("bf16", 8, 1, 128, 32), ("bf16", 2, 1, 64, 16), ("bf16", 3, 1, 64, 48),
        ("bf16", 4, 2, 128, 16), ("bf16", 1, 8, 64, 16), ("bf16", 2, 3, 128, 16), ("bf16", 7, 1, 128, 16), ("bf16", 4, 5, 128, 16), ("bf16", 2, 8, 64, 16), ("bf16", 8, 3, 128, 32), ("bf16", 3, 5, 64, 16), ("bf16", 4, 8, 128, 16),
        ("f32", 3, 1, 64, 16), ("f32", 7, 1, 128, 48), ("f32", 1, 1, 64, 16), ("f32", 4, 1, 128, 16), ("f32", 8, 1, 64, 32), ("f32", 2, 1, 128, 16)]
PLAIN = [("bf16", 16, 1, 128, 16), ("bf16", 5, 8, 128, 16), ("bf16", 4, 1, 96, 16), ("bf16", 1, 1, 128, 10), ("f32", 9, 1, 64, 16),
         ("f32", 2, 2, 128, 16), ("f32", 1, 1, 256, 1), ("bf16", 5, 8, 7, 3), ("f32", 4, 1, 33, 17)]


def half_step(dtype):
    return 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24


class Run:
    def __init__(self, shape, lens, hkv=2, seed=0, gain=1.0):
        self.dtype, self.group, self.Q, self.D, self.bs = shape
        self.cache = c = ref.Cache(lens, hkv, self.D, self.dtype, self.bs, seed)
        self.q = c.queries(self.Q, self.group * hkv, gain)
        self.scale = self.D ** -0.5
        self.hkv, self.lens = hkv, list(lens)
        self.table = torch.from_numpy(c.table).cuda()
        self.n = torch.tensor(self.lens, dtype=torch.int32).cuda()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.dq = c.upload(self.q)
        self.dk, self.dv = c.upload(c.place(c.k)), c.upload(c.place(c.v))
        self.bound = max(1, max(lens))

    def out(self):
        return torch.full_like(self.dq, 7.0)

    def sinks(self, window, sinks, **kw):
        o = self.out()
        pkg.pa_decode_sinks(self.dq, self.dk, self.dv, self.table, self.n, self.scale, window, sinks, o, self.bound, error_word=self.err, **kw)
        return o.double().cpu().numpy()

    def weights(self, start, **kw):
        o, w = self.out(), torch.from_numpy(start).cuda()
        pkg.pa_decode_weights(self.dq, self.dk, self.dv, self.table, self.n, self.scale, o, w, self.bound, error_word=self.err, **kw)
        return o.double().cpu().numpy(), w.cpu().numpy()

    def check(self, got, window=0, sinks=0, only=None):
        for s, n in enumerate(self.lens):
            want, _, tol, _ = ref.attention(self.q[s], self.cache.k[s], self.cache.v[s], self.scale, self.group, window, sinks, self.dtype == "bf16")
            off = np.abs(got[s] - want)
            ok = off <= tol + half_step(self.dtype) * (np.abs(want) + tol) + 1e-30
            assert ok[only if only is not None else slice(None)].all(), (s, n, window, sinks, np.nanmax(off), off.shape)


def lens_for(Q):
    return [0, Q, Q + 1, 15 + Q, 17 + Q, 64, 511, 512, 513, 1100, 1551]


@pytest.mark.parametrize("shape", RING + PLAIN, ids=str)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 4), (16, 16), (64, 4), (200, 33), (512, 64), (1024, 600), (100000, 4)])
def test_sinks(shape, window, sinks):
    run = Run(shape, lens_for(shape[2]), seed=window + sinks)
    run.check(run.sinks(window, sinks), window, sinks)
    assert int(run.err.item()) == 0


@pytest.mark.parametrize("shape", RING + PLAIN, ids=str)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_rows_that_no_token_sees_may_hold_anything(shape, bad):
    window, sinks = 40, 21
    Q = shape[2]
    run = Run(shape, lens_for(Q), seed=5)
    c = run.cache
    k, v = [x.copy() for x in c.k], [x.copy() for x in c.v]
    for s, n in enumerate(run.lens):
        seen = set().union(*(set(ref.visible(n, Q, j, window, sinks)) for j in range(Q))) if n else set()
        for i in set(range(n)) - seen:
            k[s][i], v[s][i] = bad, bad
    run.dk, run.dv = c.upload(c.place(k, bad)), c.upload(c.place(v, bad))
    run.check(run.sinks(window, sinks), window, sinks)


@pytest.mark.parametrize("shape", [s for s in RING + PLAIN if s[2] > 1], ids=str)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("window,sinks", [(5, 0), (40, 21), (700, 3)])
def test_a_row_reaches_only_the_tokens_that_see_it(shape, bad, window, sinks):
    """The last row is seen by the last token alone, the row that has just left the
    other tokens' windows by the first."""
    Q = shape[2]
    lens = [Q + window + 30, 600 + window, Q + 1]
    for place, clean in ((lambda n: n - 1, slice(0, Q - 1)), (lambda n: n - Q - window + 1, slice(1, Q))):
        run = Run(shape, lens, seed=6)
        c = run.cache
        for s, n in enumerate(lens):
            if place(n) >= sinks:
                run.dk[c.table[s, place(n) // c.bs], :, place(n) % c.bs] = bad
                run.dv[c.table[s, place(n) // c.bs], :, place(n) % c.bs] = bad
        run.check(run.sinks(window, sinks), window, sinks, only=clean)


def start_weights(cache, seed=3):
    return np.random.default_rng(seed).gamma(0.5, 2.0, (cache.num_blocks, cache.hkv, cache.bs)).astype(np.float32)


def check_weights(run, start, got, calls=1):
    c = run.cache
    left = np.ones_like(start, bool)
    for s, n in enumerate(run.lens):
        if n == 0:
            continue
        _, w, _, tol = ref.attention(run.q[s], c.k[s], c.v[s], run.scale, run.group)
        old = ref.slot_rows(start, c.table[s], n, c.bs).astype(np.float64)
        new = np.arange(n)[:, None] >= n - run.Q
        want = np.where(new, w, old + calls * w)
        off = np.abs(ref.slot_rows(got, c.table[s], n, c.bs) - want)
        assert (off <= calls * (tol + 2.0 ** -24 * (want + tol))).all(), (s, n, off.max())
        i = np.arange(n)
        left[c.table[s, i // c.bs], :, i % c.bs] = False
    assert np.array_equal(got[left], start[left])         # rows of nobody


@pytest.mark.parametrize("shape", RING + PLAIN, ids=str)
@pytest.mark.parametrize("gain", [1.0, 4.0])
def test_weights(shape, gain):
    run = Run(shape, lens_for(shape[2]), seed=9, gain=gain)
    start = start_weights(run.cache)
    for s, n in enumerate(run.lens):                   # what a new row's slot held does not matter
        for i in range(max(0, n - run.Q), n):
            start[run.cache.table[s, i // run.bs], :, i % run.bs] = np.nan
    out, got = run.weights(start)
    run.check(out)
    check_weights(run, start, got)
    assert int(run.err.item()) == 0


def test_weights_add_up_to_the_tokens_and_heads():
    """Over a sequence the weights of one call add up to heads per KV head x tokens."""
    run = Run(("bf16", 4, 2, 128, 16), [1300, 40, 2], seed=1)
    _, got = run.weights(np.zeros((run.cache.num_blocks, run.hkv, run.bs), np.float32))
    for s, n in enumerate(run.lens):
        total = ref.slot_rows(got, run.cache.table[s], n, run.bs).astype(np.float64).sum(0)
        assert np.abs(total - 8).max() <= 8 * 2.0 ** -13


def test_weights_of_a_shared_block_are_those_of_both_sequences():
    run = Run(("bf16", 4, 1, 128, 16), [100, 100], seed=2)
    c = run.cache
    c.table[1, :3] = c.table[0, :3]                    # rows 0 .. 47 shared, as after a fork
    for x in (c.k, c.v):
        x[1][:48] = x[0][:48]
    run.table = torch.from_numpy(c.table).cuda()
    run.dk, run.dv = c.upload(c.place(c.k)), c.upload(c.place(c.v))
    _, got = run.weights(np.zeros((c.num_blocks, run.hkv, run.bs), np.float32))
    each = [ref.attention(run.q[s], c.k[s], c.v[s], run.scale, run.group)[1::2] for s in (0, 1)]
    want, tol = each[0][0][:48] + each[1][0][:48], each[0][1][:48] + each[1][1][:48]
    assert (np.abs(ref.slot_rows(got, c.table[0], 48, 16) - want) <= tol + 2.0 ** -23 * want).all()


@pytest.mark.parametrize("shape", [RING[1], RING[5], RING[9], RING[-1], PLAIN[1], PLAIN[4]], ids=str)
def test_flagged_sequences_are_left_out(shape):
    Q = shape[2]
    run = Run(shape, [600, 40, 530, 70, 33], seed=4)
    if Q > 1:
        run.n[1] = Q - 1                               # fewer rows than tokens
    else:
        run.n[1] = -1
    run.n[3] = run.bound + 1
    run.table[2, 31] = run.cache.num_blocks            # outside the pool (rows 496 ..)
    start = start_weights(run.cache)
    out, got = run.weights(start)
    assert int(run.err.item()) == pa.PA_DEVERR_CONTEXT | pa.PA_DEVERR_BLOCK_ID
    for s in (1, 2, 3):
        n, b = run.lens[s], run.cache.table[s]
        assert np.array_equal(ref.slot_rows(got, b, n, run.bs), ref.slot_rows(start, b, n, run.bs))
    run.err.zero_()
    outs = run.sinks(64, 4)
    assert int(run.err.item()) in (pa.PA_DEVERR_CONTEXT | pa.PA_DEVERR_BLOCK_ID, pa.PA_DEVERR_CONTEXT)
    for got, window, sinks in ((out, 0, 0), (outs, 64, 4)):
        for s in (0, 4):
            want, _, tol, _ = ref.attention(run.q[s], run.cache.k[s], run.cache.v[s], run.scale, run.group, window, sinks, run.dtype == "bf16")
            assert (np.abs(got[s] - want) <= tol + half_step(run.dtype) * (np.abs(want) + tol)).all()


@pytest.mark.parametrize("shape", [RING[1], RING[5], RING[9], RING[-1], PLAIN[0], PLAIN[4]], ids=str)
def test_a_sequence_does_not_depend_on_the_rest_of_the_batch(shape):
    run = Run(shape, [1551, 40, 700, 0, 513, 1024, 9, 8], seed=11)
    start = start_weights(run.cache)
    whole = [run.sinks(300, 20), *run.weights(start)]
    for s in (0, 2, 4):
        one = Run(shape, [1551, 40, 700, 0, 513, 1024, 9, 8], seed=11)
        one.dq, one.table, one.n = one.dq[s:s + 1], one.table[s:s + 1], one.n[s:s + 1]
        assert np.array_equal(one.sinks(300, 20)[0], whole[0][s])
        out, got = one.weights(start)
        assert np.array_equal(out[0], whole[1][s])
        n = run.lens[s]
        assert np.array_equal(ref.slot_rows(got, run.cache.table[s], n, run.bs), ref.slot_rows(whole[2], run.cache.table[s], n, run.bs))


def test_more_sequences_than_a_launch_holds():
    r = np.random.default_rng(0)
    lens = [int(x) for x in r.integers(0, 40, 4100)] + [700]
    run = Run(("bf16", 2, 1, 64, 16), lens, hkv=1, seed=12)
    run.check(run.sinks(9, 2), 9, 2)
    start = start_weights(run.cache)
    out, got = run.weights(start)
    run.check(out)
    check_weights(run, start, got)


def test_a_window_that_holds_every_row_is_none():
    run = Run(("bf16", 4, 1, 128, 16), [1551, 512, 7, 0], seed=13)
    for got in (run.sinks(1551, 0), run.sinks(2 ** 31 - 1, 2 ** 31 - 1), run.weights(start_weights(run.cache))[0]):
        run.check(got)
    # Windows of 1,000 rows lie in partitions of 512, as decoding without one has them: the same bits.
    run = Run(("bf16", 4, 1, 128, 16), [991, 512, 7, 0], seed=13)
    assert np.array_equal(run.weights(start_weights(run.cache))[0], run.sinks(1000, 0))


@pytest.mark.parametrize("shape", [RING[1], RING[5], RING[11], RING[-1], PLAIN[2]], ids=str)
def test_captured_and_replayed(shape):
    """Both calls in one graph over one workspace, replayed with other queries."""
    run = Run(shape, [900, 64, 0, 513], seed=14)
    hq = run.group * run.hkv
    need = max(pkg.pa_decode_workspace_size_weights(4, run.Q, hq, run.D, run.bound), pa.pa_decode_workspace_size_multi(4, run.Q, hq, run.D, run.bound))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    start = start_weights(run.cache)
    o1, o2, w = run.out(), run.out(), torch.from_numpy(start).cuda()
    args = (run.dq, run.dk, run.dv, run.table, run.n, run.scale)

    def both():
        pkg.pa_decode_sinks(*args, 100, 4, o1, run.bound, workspace=ws, error_word=run.err)
        pkg.pa_decode_weights(*args, o2, w, run.bound, workspace=ws, error_word=run.err)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    run.q = run.cache.queries(run.Q, hq)
    run.dq.copy_(run.cache.upload(run.q))
    w.copy_(torch.from_numpy(start))
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    run.check(o1.double().cpu().numpy(), 100, 4)
    run.check(o2.double().cpu().numpy())
    check_weights(run, start, w.cpu().numpy(), calls=2)


def test_on_another_stream_with_scratch_of_its_own():
    run = Run(("bf16", 4, 1, 128, 16), [900, 64, 513], seed=15)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = run.out()
    torch.cuda.synchronize()
    pkg.pa_decode_sinks(run.dq, run.dk, run.dv, run.table, run.n, run.scale, 77, 3, o, run.bound, stream=side)
    side.synchronize()
    run.check(o.double().cpu().numpy(), 77, 3)


@pytest.mark.parametrize("shape", RING, ids=str)
def test_weights_of_short_sequences(shape):
    """Sequences of one partition each: as in 64 bits, flagged ones left out, and the bits of the
    same call with a length bound that allows more partitions."""
    Q = shape[2]
    lens = [0, Q, Q + 1, 15 + Q, 17 + Q, 64, 511, 512, 300, 90]
    run = Run(shape, lens, seed=15)
    start = start_weights(run.cache)
    out, got = run.weights(start)
    run.check(out)
    check_weights(run, start, got)
    run.table = torch.nn.functional.pad(run.table, (0, 1), value=-1)
    run.bound = 513
    for a, b in zip(run.weights(start), (out, got)):
        assert np.array_equal(a, b)
    run.bound = 512
    run.n[8] = Q - 1 if Q > 1 else -1
    run.n[9] = run.bound + 1
    run.table[7, 1] = run.cache.num_blocks
    out1, got1 = run.weights(start)
    assert int(run.err.item()) == pa.PA_DEVERR_CONTEXT | pa.PA_DEVERR_BLOCK_ID
    for s, n in enumerate(lens):
        rows = lambda w: ref.slot_rows(w, run.cache.table[s], n, run.bs)
        assert np.array_equal(rows(got1), rows(start if s in (7, 8, 9) else got))
        assert s in (7, 8, 9) or np.array_equal(out1[s], out[s])


@pytest.mark.parametrize("shape", [RING[1], RING[3], RING[-1]], ids=str)
def test_short_sequences_alone_and_in_a_large_batch(shape):
    r = np.random.default_rng(3)
    lens = [int(x) for x in r.integers(1, 60, 700)] + [512]
    run = Run(shape, lens, seed=16)
    start = start_weights(run.cache)
    out, got = run.weights(start)
    run.check(out)
    check_weights(run, start, got)
    dq, table, n = run.dq, run.table, run.n
    for a, b in ((0, 1), (40, 300), (600, 701)):
        run.dq, run.table, run.n = dq[a:b], table[a:b], n[a:b]
        out1, got1 = run.weights(start)
        assert np.array_equal(out1, out[a:b])
        for s in range(a, b):
            assert np.array_equal(*(ref.slot_rows(w, run.cache.table[s], lens[s], run.bs) for w in (got1, got)))


@pytest.mark.parametrize("shape", [RING[1], RING[5], RING[-1], PLAIN[0], PLAIN[4]], ids=str)
@pytest.mark.parametrize("window,sinks", [(700, 4), (660, 0), (1024, 4), (30, 2000), (1600, 100)])
def test_a_sequence_does_not_depend_on_the_bound_of_the_lengths(shape, window, sinks):
    """Also where no row can be outside the window, or the first rows are all there are."""
    run = Run(shape, [690, 40, 600, 513], seed=17)
    run.table = torch.nn.functional.pad(run.table, (0, 5000 // shape[4] + 1), value=-1)
    want = run.sinks(window, sinks)
    for bound in (701, 752, 1025, 2500, 5000):
        run.bound = bound
        assert np.array_equal(run.sinks(window, sinks), want)
    assert int(run.err.item()) == 0
