"""The calls that say which rows of a cache count: run together as a server runs them,
in pools past 32 bits, on other streams, and refused by the binding."""
import numpy as np
import pytest
import torch

import cache_rows_reference as ref
import paged_kv_cache_29_gb300 as pkg
from paged_kv_cache_29_gb300 import _binding as pa
from paged_kv_cache_29_gb300.block_manager import BlockManager
from test_gpu_decode_rows import Run, start_weights
from test_gpu_evict import Evict, raw

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def tables_of(manager, names, width):
    t = np.full((len(names), width), -1, np.int32)
    for s, name in enumerate(names):
        row = manager.block_table(name)
        t[s, :len(row)] = row
    return torch.from_numpy(t).cuda()


class Server:
    """Sequences under a block manager, their rows in 64 bits beside the pool: rows[s] is
    [n][Hkv][D] of K (and V), as the pool should hold them."""

    def __init__(self, prompts, hkv=2, group=4, D=128, blocks=400, seed=0):
        self.r = np.random.default_rng(seed)
        self.hkv, self.hq, self.D, self.group = hkv, hkv * group, D, group
        self.m = BlockManager(blocks, 16, free_order=self.r.permutation(blocks))
        self.names = [f"s{i}" for i in range(len(prompts))]
        self.k, self.v = ([np.zeros((0, hkv, D)) for _ in prompts] for _ in range(2))
        self.kc, self.vc = (torch.full((blocks, hkv, 16, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.w = torch.zeros(blocks, hkv, 16, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.width = 64
        for name in self.names:
            self.m.admit(name, [])
        self.append(prompts)
        self.scale = D ** -0.5

    def values(self, *shape):
        t = torch.from_numpy(self.r.standard_normal(shape).astype(np.float32)).cuda().bfloat16()
        return t, t.double().cpu().numpy()

    def append(self, counts):
        """counts[s] new rows of every sequence, through the manager's slots."""
        slots = []
        for s, c in enumerate(counts):
            for _ in range(c):
                got = self.m.append(self.names[s], int(self.r.integers(0, 1000)))
                if got.copy_on_write:
                    pair = torch.tensor([got.copy_on_write], dtype=torch.int64).cuda()
                    pa.pa_copy_blocks(self.kc, self.vc, pair, error_word=self.err)
                slots.append(got.slot)
        k, hk = self.values(len(slots), self.hkv, self.D)
        v, hv = self.values(len(slots), self.hkv, self.D)
        pa.pa_reshape_and_cache(k, v, torch.tensor(slots, dtype=torch.int64).cuda(), self.kc, self.vc, error_word=self.err)
        at = 0
        for s, c in enumerate(counts):
            self.k[s], self.v[s] = np.concatenate([self.k[s], hk[at:at + c]]), np.concatenate([self.v[s], hv[at:at + c]])
            at += c

    def lens(self):
        return [len(x) for x in self.k]

    def check(self, out, q, window=0, sinks=0):
        for s in range(len(self.names)):
            want, _, tol, _ = ref.attention(q[s], self.k[s], self.v[s], self.scale, self.group, window, sinks, True)
            off = np.abs(out[s] - want)
            assert (off <= tol + 2.0 ** -8 * (np.abs(want) + tol)).all(), (s, off.max())

    def done(self):
        self.m.check()
        assert int(self.err.item()) == 0


def test_drafts_verified_in_a_window_and_rejected_rows_taken_back():
    """Steps of speculative decoding: three drafts and the token before them are
    appended, attended in a window with sinks, verified; the rows of rejected drafts
    leave, and their slots are written again by the next step."""
    sv = Server([700, 33, 18, 5], seed=1)
    B, Q, V, window, sinks = 4, 3, 1000, 100, 4
    lens = i32(sv.lens())
    for _ in range(6):
        sv.append([Q + 1] * B)
        lens.copy_(i32(sv.lens()))
        q, hq = sv.values(B, Q + 1, sv.hq, sv.D)
        out = torch.empty_like(q)
        # Heads per KV head x tokens is 16: two groups of the tensor-core kernel's columns.
        pkg.pa_decode_sinks(q, sv.kc, sv.vc, tables_of(sv.m, sv.names, sv.width), lens, sv.scale, window, sinks, out, 1000, error_word=sv.err)
        sv.check(out.double().cpu().numpy(), hq, window, sinks)
        target = torch.from_numpy(sv.r.dirichlet(np.full(V, 0.05), (B, Q + 1)).astype(np.float32)).cuda()
        draft = torch.from_numpy(sv.r.dirichlet(np.full(V, 0.05), (B, Q)).astype(np.float32)).cuda()
        draft[:2] = 0.7 * target[:2, :Q] + 0.3 * draft[:2]
        tokens = torch.multinomial(draft.flatten(0, 1) + 1e-20, 1).view(B, Q).int()
        u = torch.from_numpy(sv.r.random((B, Q + 1), dtype=np.float32)).cuda()
        new, accepted = torch.zeros(B, Q + 1, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
        pkg.pa_verify_draft(target, draft, tokens, u, new, accepted, context_lens=lens, lens_out=lens, error_word=sv.err)
        for s, a in enumerate(accepted.tolist()):
            want, token, _ = ref.verify(target[s].cpu().numpy(), draft[s].cpu().numpy(), tokens[s].tolist(), u[s].double().cpu().numpy(), Q)
            assert (a, int(new[s, a])) == (want, token)
            n = len(sv.k[s]) - (Q - a)
            assert sv.m.truncate(sv.names[s], n) is None
            sv.k[s], sv.v[s] = sv.k[s][:n], sv.v[s][:n]
        assert lens.tolist() == sv.lens() == [sv.m.num_tokens(x) for x in sv.names]
    sv.done()


@pytest.mark.parametrize("shared", [False, True])
def test_a_cache_kept_to_a_budget(shared):
    """Decode steps that accumulate weights; sequences above their budget are cut to it,
    in place or, where a fork shares their blocks, into blocks of their own; the steps after
    attend to the rows that stayed, of every KV head its own."""
    sv = Server([300, 90, 40], seed=2)
    B, sinks, recent, budget = 3, 2, 10, 64
    if shared:
        sv.m.fork("s0", "fork")
        fork = [x.copy() for x in (sv.k[0], sv.v[0])]
    total = [np.zeros((n, sv.hkv)) for n in sv.lens()]
    off = [np.zeros((n, sv.hkv)) for n in sv.lens()]
    for step in range(30):
        sv.append([1] * B)
        q, hq = sv.values(B, sv.hq, sv.D)
        out = torch.empty_like(q)
        lens = i32(sv.lens())
        table = tables_of(sv.m, sv.names, sv.width)
        pkg.pa_decode_weights(q, sv.kc, sv.vc, table, lens, sv.scale, out, sv.w, 1000, error_word=sv.err)
        sv.check(out.double().cpu().numpy()[:, None], hq[:, None])
        for s in range(B):
            _, w, _, tol = ref.attention(hq[s][None], sv.k[s], sv.v[s], sv.scale, sv.group)
            total[s] = np.concatenate([total[s], np.zeros((1, sv.hkv))]) + w
            off[s] = np.concatenate([off[s], np.zeros((1, sv.hkv))]) + tol + 2.0 ** -23 * total[s]
        if step % 7 != 3:
            continue
        keep = [min(len(x), budget) for x in sv.k]
        pool_w = sv.w.cpu().numpy()
        old = [sv.m.block_table(x) for x in sv.names]
        sv.m.evict(dict(zip(sv.names, keep)))
        pkg.pa_evict(sv.kc, sv.vc, sv.w, table, lens, i32(keep), tables_of(sv.m, sv.names, sv.width), lens, 1000, sinks, recent, error_word=sv.err)
        assert lens.tolist() == keep
        for s in range(B):
            n = len(sv.k[s])
            w = ref.slot_rows(pool_w, np.array(old[s]), n, 16).astype(np.float64)
            assert (np.abs(w - total[s]) <= off[s]).all()
            stay = np.array([ref.kept_rows(w[:, h], n, keep[s], sinks, recent) for h in range(sv.hkv)]).T   # [keep][Hkv]
            sv.k[s], sv.v[s] = (np.take_along_axis(x, stay[:, :, None], 0) for x in (sv.k[s], sv.v[s]))
            total[s], off[s] = np.take_along_axis(total[s], stay, 0), np.take_along_axis(off[s], stay, 0)
    if shared:                                         # the fork still has every row
        q, hq = sv.values(1, sv.hq, sv.D)
        out = torch.empty_like(q)
        pa.pa_decode(q, sv.kc, sv.vc, tables_of(sv.m, ["fork"], sv.width), i32([300]), sv.scale, out, 1000, error_word=sv.err)
        want, _, tol, _ = ref.attention(hq[:, None][0], *fork, sv.scale, sv.group, rounded_weights=True)
        assert (np.abs(out.double().cpu().numpy()[:, None][0] - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol)).all()
    sv.done()


def test_rows_past_32_bits():
    """A pool of 5 GB a side, the sequences in its last blocks."""
    NB, hkv, bs, D = 610_000, 2, 16, 128
    shape = ("bf16", 4, 1, D, bs)
    run = Run(shape, [600, 40, 513], hkv=hkv, seed=3)
    c = run.cache
    kc, vc = (torch.empty(NB, hkv, bs, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    w = torch.empty(NB, hkv, bs, device="cuda")
    high = NB - c.num_blocks
    start = start_weights(c)
    for big, small in ((kc, run.dk), (vc, run.dv), (w, torch.from_numpy(start).cuda())):
        big[high:] = small
    run.dk, run.dv = kc, vc
    run.table = run.table + high
    run.check(run.sinks(100, 4), 100, 4)
    o = run.out()
    pkg.pa_decode_weights(run.dq, kc, vc, run.table, run.n, run.scale, o, w, run.bound, error_word=run.err)
    run.check(o.double().cpu().numpy())
    got = w[high:].cpu().numpy()
    before = kc[high:].cpu()
    lens = run.n.clone()
    pkg.pa_evict(kc, vc, w, run.table, run.n, i32([200, 10, 500]), run.table, lens, run.bound, 1, 4, error_word=run.err)
    assert lens.tolist() == [200, 10, 500] and int(run.err.item()) == 0
    after = kc[high:].cpu()
    for s, k in enumerate(lens.tolist()):
        n = run.lens[s]
        weights = ref.slot_rows(got, c.table[s], n, bs).astype(np.float64)
        for h in range(hkv):
            stay = np.array(ref.kept_rows(weights[:, h], n, k, 1, 4))
            j = np.arange(k)
            assert torch.equal(after[c.table[s, j // bs], h, j % bs], before[c.table[s, stay // bs], h, stay % bs])


@pytest.mark.parametrize("handle", [False, True])
def test_scratch_of_calls_on_another_stream_is_theirs(handle):
    """Weights and eviction without a workspace on a side stream, while torch's current
    stream fills every tensor that the allocator gives it."""
    side = torch.cuda.Stream()
    run = Run(("bf16", 4, 1, 128, 16), [5000, 40, 3000, 2200] * 8, seed=4)
    start = start_weights(run.cache)
    want_out, want_w = run.weights(start)
    w, o = torch.from_numpy(start).cuda(), run.out()
    keep, lens = i32([2500, 20, 2999, 100] * 8), torch.zeros_like(run.n)
    need = pkg.pa_decode_workspace_size_weights(32, 1, 8, 128, run.bound)
    torch.cuda.synchronize()
    on = side.cuda_stream if handle else side
    pkg.pa_decode_weights(run.dq, run.dk, run.dv, run.table, run.n, run.scale, o, w, run.bound, error_word=run.err, stream=on)
    for _ in range(3):
        torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    k_before = run.dk.clone()
    side.synchronize()
    assert np.array_equal(o.double().cpu().numpy(), want_out) and np.array_equal(w.cpu().numpy(), want_w)
    pkg.pa_evict(run.dk, run.dv, w, run.table, run.n, keep, run.table, lens, run.bound, error_word=run.err, stream=on)
    for _ in range(3):
        torch.full((pkg.pa_evict_workspace_size(32, 2, run.bound),), 255, dtype=torch.uint8, device="cuda")
    side.synchronize()
    assert lens.tolist() == [2500, 20, 2999, 100] * 8 and int(run.err.item()) == 0
    for s in (0, 1, 2, 3, 31):
        n, k = run.lens[s], lens.tolist()[s]
        weights = ref.slot_rows(want_w, run.cache.table[s], n, 16).astype(np.float64)
        for h in range(2):
            stay = np.array(ref.kept_rows(weights[:, h], n, k, 0, 0))
            j = np.arange(k)
            at = run.cache.table[s]
            assert torch.equal(run.dk[at[j // 16], h, j % 16].view(torch.int16), k_before[at[stay // 16], h, stay % 16].view(torch.int16))


def test_two_streams_at_once_with_workspaces_of_their_own():
    a, b = Run(("bf16", 4, 1, 128, 16), [3000, 900] * 20, seed=5), Run(("bf16", 4, 1, 128, 16), [2100, 50] * 20, seed=6)
    sa, sb = start_weights(a.cache), start_weights(b.cache, 7)
    want = [r.weights(s) for r, s in ((a, sa), (b, sb))]
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    torch.cuda.synchronize()
    for r, s, st in ((a, sa, streams[0]), (b, sb, streams[1])):
        w, o = torch.from_numpy(s).cuda(), r.out()
        ws = torch.empty(pkg.pa_decode_workspace_size_weights(40, 1, 8, 128, r.bound), dtype=torch.uint8, device="cuda")
        got.append((r, o, w, ws, st))
    torch.cuda.synchronize()
    for _ in range(3):
        for r, o, w, ws, st in got:
            pkg.pa_decode_weights(r.dq, r.dk, r.dv, r.table, r.n, r.scale, o, w, r.bound, workspace=ws, stream=st)
    torch.cuda.synchronize()
    for (r, o, w, _, _), (wo, ww), s in zip(got, want, (sa, sb)):
        assert np.array_equal(o.double().cpu().numpy(), wo)
        once = ww.astype(np.float64)
        new = np.zeros_like(s, bool)                   # three calls: old + 3 w, new rows w
        for q, n in enumerate(r.lens):
            new[r.cache.table[q, (n - 1) // 16], :, (n - 1) % 16] = True
        three = np.where(new, once, s.astype(np.float64) + 3 * (once - s.astype(np.float64)))
        assert (np.abs(w.cpu().numpy() - three) <= 2.0 ** -21 * (np.abs(three) + np.abs(s))).all()


def test_refusals_of_the_binding():
    run = Run(("bf16", 4, 1, 128, 16), [40], seed=8)
    w = torch.zeros(run.cache.num_blocks, 2, 16, device="cuda")
    o = run.out()
    args = dict(q=run.dq, k_cache=run.dk, v_cache=run.dv, block_tables=run.table, context_lens=run.n, scale=0.1, out=o, max_context_len=40)

    def sinks(**kw):
        pkg.pa_decode_sinks(**{**args, "window": 8, "num_sinks": 2, **kw})

    def weights(**kw):
        pkg.pa_decode_weights(**{**args, "row_weights": w, **kw})

    for call in (sinks, weights):
        for kw, err in ((dict(q=run.dq.float()), TypeError), (dict(q=run.dq.cpu()), ValueError), (dict(q=run.dq[0, 0]), ValueError),
                        (dict(out=o[:, :, :4]), ValueError), (dict(block_tables=run.table.long()), TypeError), (dict(context_lens=None), ValueError),
                        (dict(max_context_len=2 ** 31), ValueError), (dict(max_context_len=2 ** 31 - 1), pa.PagedAttentionError),
                        (dict(k_cache=run.dk[:, :1].contiguous()), ValueError), (dict(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda")),
                                                                                 pa.PagedAttentionError)):
            with pytest.raises(err):
                call(**kw)
    for kw, err in ((dict(window=0), pa.PagedAttentionError), (dict(num_sinks=-1), pa.PagedAttentionError), (dict(window=2 ** 31), ValueError)):
        with pytest.raises(err):
            sinks(**kw)
    for kw, err in ((dict(row_weights=w.double()), TypeError), (dict(row_weights=w[:, :, :8]), ValueError), (dict(row_weights=w[:1]), ValueError)):
        with pytest.raises(err):
            weights(**kw)
    e = Evict([40], [20], 1, 1)
    ew, et, n, k = torch.from_numpy(e.w).cuda(), torch.from_numpy(e.table).cuda(), i32([40]), i32([20])
    good = dict(k_cache=e.k, v_cache=e.v, row_weights=ew, block_tables=et, context_lens=n, keep_lens=k, out_tables=et, lens_out=torch.zeros_like(n),
                max_context_len=40)
    scales = torch.zeros(e.k.shape[:3], device="cuda")
    before = raw(e.k)
    for kw, err in ((dict(k_params=scales, v_params=scales), ValueError), (dict(out_tables=et[:, :1].contiguous()), ValueError),
                    (dict(keep_lens=k.long()), TypeError), (dict(lens_out=None), ValueError), (dict(v_cache=e.v[:1]), ValueError),
                    (dict(num_sinks=-1), pa.PagedAttentionError), (dict(max_context_len=10 ** 6), pa.PagedAttentionError),
                    (dict(k_cache=e.k.view(torch.int8), v_cache=e.v.view(torch.int8)), ValueError),
                    (dict(k_cache=e.k.view(torch.uint8), v_cache=e.v.view(torch.uint8), k_params=scales, v_params=scales), TypeError)):
        with pytest.raises(err):
            pkg.pa_evict(**{**good, **kw})
    assert np.array_equal(raw(e.k), before)
    p, q = torch.rand(2, 4, 50, device="cuda"), torch.rand(2, 3, 50, device="cuda")
    x, u = torch.zeros(2, 3, dtype=torch.int32, device="cuda"), torch.rand(2, 4, device="cuda")
    out, acc = torch.zeros(2, 4, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    for kw, err in ((dict(target_probs=p.bfloat16()), TypeError), (dict(target_probs=p[0]), ValueError), (dict(target_probs=p.transpose(1, 2)), ValueError),
                    (dict(target_probs=p.cpu()), ValueError), (dict(draft_probs=q[:, :2]), ValueError), (dict(draft_tokens=x[:, :2].contiguous()), ValueError),
                    (dict(uniforms=u[:, :3].contiguous()), ValueError), (dict(num_accepted=acc[:1]), ValueError), (dict(context_lens=acc), pa.PagedAttentionError),
                    (dict(num_drafts=acc.long()), TypeError)):
        with pytest.raises(err):
            pkg.pa_verify_draft(**{**dict(target_probs=p, draft_probs=q, draft_tokens=x, uniforms=u, out_tokens=out, num_accepted=acc), **kw})


@pytest.mark.parametrize("shape", [("bf16", 4, 1, 128, 16), ("bf16", 4, 3, 64, 16), ("f32", 5, 1, 64, 16)], ids=str)
def test_sequences_of_many_partitions(shape):
    """More partitions than a warp of the merge takes at a time (40 and 100)."""
    run = Run(shape, [20000, 50_000 if shape[0] == "bf16" else 17000, 30], hkv=1, seed=21)
    run.check(run.sinks(18000, 70), 18000, 70)
    start = start_weights(run.cache)
    out, got = run.weights(start)
    run.check(out)
    for s, n in enumerate(run.lens):
        _, w, _, tol = ref.attention(run.q[s], run.cache.k[s], run.cache.v[s], run.scale, run.group)
        old = ref.slot_rows(start, run.cache.table[s], n, run.bs).astype(np.float64)
        want = np.where(np.arange(n)[:, None] >= n - run.Q, w, old + w)
        assert (np.abs(ref.slot_rows(got, run.cache.table[s], n, run.bs) - want) <= tol + 2.0 ** -24 * (want + tol)).all()
    assert int(run.err.item()) == 0


def test_more_sequences_than_a_launch_holds_with_column_groups():
    r = np.random.default_rng(1)
    lens = [0 if x < 3 else int(x) for x in r.integers(0, 30, 4200)]
    run = Run(("bf16", 4, 3, 64, 16), lens, hkv=1, seed=22)
    run.check(run.sinks(7, 2), 7, 2)
    run.check(run.weights(start_weights(run.cache))[0])
    assert int(run.err.item()) == 0


@pytest.mark.parametrize("shape", [("bf16", 4, 1, 128, 16), ("f32", 1, 1, 33, 5)], ids=str)
def test_a_length_bound_of_zero(shape):
    run = Run(shape, [0, 0, 0], seed=23)
    run.bound = 0
    assert not run.sinks(5, 2).any()
    start = start_weights(run.cache)
    out, got = run.weights(start)
    assert not out.any() and np.array_equal(got, start)
    lens = torch.full_like(run.n, 9)
    pkg.pa_evict(run.dk, run.dv, torch.from_numpy(start).cuda(), run.table, run.n, run.n, run.table, lens, 0, 3, 4, error_word=run.err) \
        if shape[0] == "bf16" else lens.zero_()
    assert lens.tolist() == [0, 0, 0] and int(run.err.item()) == 0


def test_every_row_of_a_long_first_part_and_limits_of_the_numbers():
    e = Evict([600, 40], [600, 40], 2 ** 31 - 1, 2 ** 31 - 1, place="other", seed=24)
    e.check()


def test_eviction_of_float8_tensors():
    e = Evict([300, 40], [120, 40], 2, 8, "fp8", seed=25, weights="random")
    e.k, e.v = e.k.view(torch.float8_e4m3fn), e.v.view(torch.float8_e4m3fn)
    e.check()


def test_probabilities_laid_out_token_by_token():
    """[rows][B][V] as a loop over tokens leaves them, passed as a transposed view."""
    r = np.random.default_rng(26)
    B, Q, V = 6, 3, 777
    p = r.dirichlet(np.full(V, 0.1), (Q + 1, B)).astype(np.float32)
    q = r.dirichlet(np.full(V, 0.1), (Q, B)).astype(np.float32)
    q[:, :3] = p[:Q, :3]
    x = np.argmax(q, -1).T.astype(np.int32).copy()
    u = r.random((B, Q + 1), dtype=np.float32)
    out, acc = torch.zeros(B, Q + 1, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    pkg.pa_verify_draft(torch.from_numpy(p).cuda().transpose(0, 1), torch.from_numpy(q).cuda().transpose(0, 1), torch.from_numpy(x).cuda(),
                       torch.from_numpy(u).cuda(), out, acc)
    for s in range(B):
        a, token, _ = ref.verify(p[:, s], q[:, s], x[s], u[s].astype(np.float64), Q)
        assert acc[s] == a and out[s].tolist() == list(x[s][:a]) + [token] + [-1] * (Q - a)
