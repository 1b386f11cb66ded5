"""pa_evict: the rows that stay, where they go, and everything else as it was."""
import numpy as np
import pytest
import torch

import cache_rows_reference as ref
import paged_kv_cache_29_gb300 as pkg
from paged_kv_cache_29_gb300 import _binding as pa

pytestmark = pytest.mark.gpu

TYPES = ["bf16", "f32", "fp8", "int8", "int4"]


def pools(r, dtype, NB, hkv, bs, D):
    """K, V and their parameters of random bytes (moved bit for bit), on the GPU."""
    bytes_ = {"bf16": 2 * D, "f32": 4 * D, "fp8": D, "int8": D, "int4": D // 2}[dtype]
    view = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.uint8, "int8": torch.int8, "int4": torch.uint8}[dtype]
    out = [torch.from_numpy(r.integers(0, 256, (NB, hkv, bs, bytes_), dtype=np.uint8)).cuda().view(view) for _ in range(2)]
    if dtype == "int8":
        out += [torch.from_numpy(r.integers(0, 256, (NB, hkv, bs, 4), dtype=np.uint8)).cuda().view(torch.float32).squeeze(-1) for _ in range(2)]
    elif dtype == "int4":
        out += [torch.from_numpy(r.integers(0, 256, (NB, hkv, bs, 4), dtype=np.uint8)).cuda().view(torch.bfloat16) for _ in range(2)]
    else:
        out += [None, None]
    return out


def raw(t):
    """The bytes of each row, [NB][Hkv][bs][...]."""
    if t is None:
        return None
    flat = t.contiguous().view(torch.uint8) if t.dim() == 4 else t.unsqueeze(-1).contiguous().view(torch.uint8)
    return flat.cpu().numpy().copy()


class Evict:
    def __init__(self, lens, keep, sinks, recent, dtype="bf16", hkv=2, D=64, bs=16, place="same", seed=0, weights="ties"):
        r = np.random.default_rng(seed)
        self.lens, self.keep, self.sinks, self.recent, self.hkv, self.bs = lens, keep, sinks, recent, hkv, bs
        need = [-(-n // bs) for n in lens]
        width = max(1, max(need))
        out_need = [-(-min(k, n) // bs) if k >= 0 else 0 for n, k in zip(lens, keep)]
        NB = sum(need) + sum(out_need) + 2
        free = [int(b) for b in r.permutation(NB)]
        self.table = np.full((len(lens), width), -1, np.int32)
        self.to = np.full((len(lens), width), -1, np.int32)
        for s, b in enumerate(need):
            self.table[s, :b] = [free.pop() for _ in range(b)]
        for s, b in enumerate(out_need):
            self.to[s, :b] = [free.pop() for _ in range(b)]
            if place == "some same":                   # the first blocks stay where they are
                half = b // 2
                self.to[s, :half] = self.table[s, :half]
        if place == "same":
            self.to = self.table.copy()
        self.k, self.v, self.kp, self.vp = pools(r, dtype, NB, hkv, bs, D)
        shape = (NB, hkv, bs)
        self.w = {"ties": lambda: r.integers(0, 6, shape).astype(np.float32), "equal": lambda: np.ones(shape, np.float32),
                  "random": lambda: r.gamma(0.3, 1.0, shape).astype(np.float32),
                  "odd": lambda: r.choice(np.float32([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, -1e-45, 3e38, -2.5, 1.0]), shape)}[weights]()
        self.bound = max(1, max(lens))

    def run(self, in_place_lens=False, same_table=False, **kw):
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        rows = [t for t in (self.k, self.v, self.kp, self.vp) if t is not None]
        before = [raw(t) for t in rows]
        w = torch.from_numpy(self.w).cuda()
        table = torch.from_numpy(self.table).cuda()
        to = table if same_table else torch.from_numpy(self.to).cuda()
        n, keep = (torch.tensor(x, dtype=torch.int32).cuda() for x in (self.lens, self.keep))
        out = n if in_place_lens else torch.full_like(n, -7)
        pkg.pa_evict(self.k, self.v, w, table, n, keep, to, out, self.bound, self.sinks, self.recent, self.kp, self.vp,
                    error_word=self.err, **kw)
        after = [raw(t) for t in rows] + [w.cpu().numpy().view(np.uint8).reshape(*self.w.shape, 4)]
        before.append(self.w.view(np.uint8).reshape(*self.w.shape, 4))
        return before, after, out.cpu().numpy()

    def check(self, flagged=(), **kw):
        before, after, out = self.run(**kw)
        want = [x.copy() for x in before]
        lens = []
        for s, n in enumerate(self.lens):
            if s in flagged:
                lens.append(n)
                continue
            k = min(n, self.keep[s])
            lens.append(k)
            w = ref.slot_rows(self.w, self.table[s], n, self.bs)
            j = np.arange(k)
            for h in range(self.hkv):
                stay = np.array(ref.kept_rows(w[:, h].astype(np.float64), n, k, self.sinks, self.recent), dtype=int)
                assert len(stay) == k
                for a, b in zip(want, before):
                    a[self.to[s, j // self.bs], h, j % self.bs] = b[self.table[s, stay // self.bs], h, stay % self.bs]
        assert list(out) == lens
        for a, b in zip(after, want):
            assert np.array_equal(a, b)
        if not flagged:
            assert int(self.err.item()) == 0


LENS = [0, 1, 5, 16, 17, 100, 255, 256, 257, 600, 1300]


def keeps(share, sinks, recent):
    return [min(n, max(int(n * share), sinks + recent)) for n in LENS]


@pytest.mark.parametrize("place", ["same", "other", "some same"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sinks,recent,share", [(0, 0, 0.5), (4, 16, 0.5), (3, 0, 0.1), (0, 33, 0.97), (1, 1, 1.0)])
def test_rows_that_stay(dtype, place, sinks, recent, share):
    Evict(LENS, keeps(share, sinks, recent), sinks, recent, dtype, place=place, seed=int(100 * share) + sinks).check()


@pytest.mark.parametrize("place", ["same", "other"])
@pytest.mark.parametrize("weights", ["equal", "random", "odd"])
@pytest.mark.parametrize("share", [0.0, 0.3, 0.999])
def test_weights_of_every_kind(weights, place, share):
    Evict(LENS, [int(n * share) for n in LENS], 0, 0, "bf16", weights=weights, place=place, seed=7).check()


@pytest.mark.parametrize("dtype,D", [("bf16", 8), ("bf16", 128), ("bf16", 256), ("f32", 256), ("f32", 4), ("f32", 100), ("int8", 16), ("int4", 32),
                                     ("int4", 256), ("int8", 240), ("fp8", 128), ("bf16", 72)])
@pytest.mark.parametrize("bs,hkv", [(16, 1), (48, 3), (1, 2), (10, 5)])
def test_shapes(dtype, D, bs, hkv):
    for place in ("same", "other"):
        Evict([300, 77, 0, 513], [150, 70, 0, 20], 2, 9, dtype, hkv=hkv, D=D, bs=bs, place=place, seed=D + bs, weights="random").check()


@pytest.mark.parametrize("place", ["same", "other"])
def test_long_sequences(place):
    """Rows beyond what one pass over the keys holds, one or a few leaving, nearly all leaving."""
    Evict([20000, 33000, 9000, 70000], [19999, 900, 8990, 40000], 4, 100, "bf16", hkv=2, D=32, place=place, seed=3, weights="random").check()


def test_in_place_of_the_lengths_and_with_one_table():
    Evict(LENS, keeps(0.4, 2, 5), 2, 5, seed=8).check(in_place_lens=True, same_table=True)


def test_many_sequences():
    r = np.random.default_rng(1)
    lens = [int(x) for x in r.integers(0, 70, 5000)]
    Evict(lens, [int(r.integers(0, n + 3)) for n in lens], 0, 0, "int8", hkv=1, D=16, seed=9, weights="random").check()


def test_a_budget_above_the_length_keeps_every_row():
    Evict([40, 7], [100, 2 ** 31 - 1], 50, 50, place="other", seed=10).check()


@pytest.mark.parametrize("place", ["same", "other"])
def test_flagged_sequences_stay_as_they_are(place):
    e = Evict([100, 90, 80, 70, 60, 50], [50, -1, 19, 35, 30, 25], 10, 10, place=place, seed=11)
    e.table[3, 2] = e.k.shape[0]                       # a block outside the pool
    if place == "other":
        e.to[4, 1] = -1
    else:
        e.to = e.table.copy()
        e.table[4, 3] = -5
        e.to[4, 3] = -5
    e.bound = 100
    before, after, out = e.run()
    assert int(e.err.item()) == pa.PA_DEVERR_CONTEXT | pa.PA_DEVERR_BLOCK_ID
    assert list(out) == [50, 90, 80, 70, 60, 25]
    for s in (1, 2):
        i = np.arange(e.lens[s])
        for a, b in zip(after, before):
            assert np.array_equal(a[e.table[s, i // 16], :, i % 16], b[e.table[s, i // 16], :, i % 16])


def test_lengths_out_of_range():
    e = Evict([100, 90, 40], [10, 10, 10], 0, 0, seed=12)
    e.bound = 90
    e.lens = [100, 90, -3]
    before, after, out = e.run()
    assert int(e.err.item()) == pa.PA_DEVERR_CONTEXT and list(out) == [100, 10, -3]


def test_captured_and_replayed_in_place():
    """A graph of an eviction in place, replayed on new contents: each replay cuts what it finds."""
    e = Evict([300, 200], [120, 64], 2, 8, seed=13, weights="random")
    w = torch.from_numpy(e.w).cuda()
    table = torch.from_numpy(e.table).cuda()
    n, keep = (torch.tensor(x, dtype=torch.int32).cuda() for x in (e.lens, e.keep))
    out = torch.zeros_like(n)
    ws = torch.empty(pkg.pa_evict_workspace_size(2, 2, 300), dtype=torch.uint8, device="cuda")
    keep_k = e.k.clone()

    def call():
        pkg.pa_evict(e.k, e.v, w, table, n, keep, table, out, 300, 2, 8, workspace=ws)

    call()
    torch.cuda.synchronize()
    first = raw(e.k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    e.k.copy_(keep_k)
    w.copy_(torch.from_numpy(e.w))
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(raw(e.k), first) and list(out.cpu()) == [120, 64]


def narrow(kind, r, shape):
    """Weights in ranges where counting passes end in parts of less than a byte's width, or of one key."""
    base = np.float32(1.0).view(np.uint32)
    spread = {"300 keys": 300, "2^12 keys": 1 << 12, "2^19 keys": 1 << 19, "one key": 1}[kind]
    bits = base + r.integers(0, spread, shape).astype(np.uint32)
    w = bits.view(np.float32)
    w[r.random(shape) < 0.05] = 0.0                    # far below the others
    return w


@pytest.mark.parametrize("kind", ["300 keys", "2^12 keys", "2^19 keys", "one key"])
@pytest.mark.parametrize("n", [600, 5000, 40000])
@pytest.mark.parametrize("place", ["same", "other"])
def test_weights_that_are_close_together(kind, n, place):
    e = Evict([n, n // 2, 3], [n // 3, n // 2 - 1, 1], 1, 0, "bf16", hkv=2, D=8, place=place, seed=n, weights="equal")
    e.w = narrow(kind, np.random.default_rng(n), e.w.shape)
    e.check()


@pytest.mark.parametrize("weights", ["random", "odd"])
def test_a_bound_beyond_what_clusters_hold(weights):
    """Lengths bounded at a million rows (the keys are read again in every pass), and one of 450,000."""
    e = Evict([450_000, 90, 0, 5000], [1000, 40, 0, 4990], 2, 20, "int4", hkv=1, D=32, place="other", seed=14, weights=weights)
    e.table = np.pad(e.table, ((0, 0), (0, 70_000 - e.table.shape[1])), constant_values=-1)
    e.to = np.pad(e.to, ((0, 0), (0, 70_000 - e.to.shape[1])), constant_values=-1)
    e.bound = 1_000_000
    e.check()


@pytest.mark.parametrize("place", ["same", "other", "some same"])
@pytest.mark.parametrize("num_seqs,hkv", [(96, 8), (255, 3), (256, 3), (257, 3)])
def test_batches_beyond_the_sms(num_seqs, hkv, place):
    """More sequences and KV heads than CTAs at a time: taken in the order of their lengths,
    up to 256 sequences; equal, empty and flagged ones among them."""
    r = np.random.default_rng(num_seqs)
    lens = [int(n) for n in r.choice([0, 1, 16, 33, 40, 40, 40, 100, 257], num_seqs)]
    lens[7], lens[30], lens[50] = 2100, 70, 333
    keep = [min(n, max(6, int(n * r.random()))) for n in lens]
    e = Evict(lens, keep, 2, 4, hkv=hkv, D=16, place=place, seed=num_seqs)
    e.check(in_place_lens=True)
    e = Evict(lens, keep, 2, 4, "int8", hkv=hkv, D=16, place=place, seed=num_seqs + 1)
    e.keep[30] = -1                                    # no length
    e.table[50, 20] = e.k.shape[0]                     # outside the pool
    e.check(flagged=(30, 50))
    assert int(e.err.item()) == pa.PA_DEVERR_CONTEXT | pa.PA_DEVERR_BLOCK_ID
    e.lens[7], e.lens[30] = -5, 2101                   # none, and above the bound
    e.check(flagged=(7, 30, 50))
