"""Row weights beside the calls that copy blocks and that take rejected rows back."""
import numpy as np
import pytest
import torch

import cache_rows_reference as ref
import paged_kv_cache_29_gb300 as pkg
from paged_kv_cache_29_gb300 import _binding as pa
from test_gpu_cache_rows_edges import Server, i32, tables_of

pytestmark = pytest.mark.gpu


def test_weights_of_a_copied_block_come_along():
    """A fork appends into a shared, partly filled block: its copy has the rows' weights too."""
    sv = Server([44], seed=61)
    start = np.random.default_rng(1).gamma(0.5, 2.0, tuple(sv.w.shape)).astype(np.float32)
    sv.w.copy_(torch.from_numpy(start))
    sv.m.fork("s0", "s1")
    source = sv.m.block_table("s0")[2]
    got = sv.m.append("s1", 7)
    assert got.copy_on_write == (source, sv.m.block_table("s1")[2])
    pair = torch.tensor([got.copy_on_write], dtype=torch.int64).cuda()
    flat = sv.w.view(sv.w.shape[0], 1, 1, -1)
    pa.pa_copy_blocks(sv.kc, sv.vc, pair, error_word=sv.err)
    pa.pa_copy_blocks(flat, flat, pair, error_word=sv.err)
    k, hk = sv.values(1, sv.hkv, sv.D)
    v, hv = sv.values(1, sv.hkv, sv.D)
    pa.pa_reshape_and_cache(k, v, torch.tensor([got.slot], dtype=torch.int64).cuda(), sv.kc, sv.vc, error_word=sv.err)
    q, hq = sv.values(1, sv.hq, sv.D)
    pkg.pa_decode_weights(q, sv.kc, sv.vc, tables_of(sv.m, ["s1"], sv.width), i32([45]), sv.scale, torch.empty_like(q), sv.w, 100, error_word=sv.err)
    _, w, _, tol = ref.attention(hq, np.concatenate([sv.k[0], hk]), np.concatenate([sv.v[0], hv]), sv.scale, sv.group)
    old = ref.slot_rows(start, np.array(sv.m.block_table("s0")), 44, 16).astype(np.float64)
    want = np.concatenate([old, np.zeros((1, sv.hkv))]) + w
    now = sv.w.cpu().numpy()
    assert (np.abs(ref.slot_rows(now, np.array(sv.m.block_table("s1")), 45, 16) - want) <= tol + 2.0 ** -24 * (want + tol)).all()
    assert np.array_equal(now[source], start[source])
    sv.m.check()
    assert int(sv.err.item()) == 0


def test_rejected_tokens_weights_stay_and_their_slots_begin_again():
    """Speculative steps that accumulate weights: every token of a step counts for the rows
    before it; the rejected ones' rows leave."""
    sv = Server([530, 40, 17], seed=62)
    B, Q, V = 3, 3, 64
    total = [np.zeros((n, sv.hkv)) for n in sv.lens()]
    off = [np.zeros((n, sv.hkv)) for n in sv.lens()]
    lens = i32(sv.lens())
    taken = 0
    for _ in range(5):
        sv.append([Q + 1] * B)
        lens.copy_(i32(sv.lens()))
        q, hq = sv.values(B, Q + 1, sv.hq, sv.D)
        out = torch.empty_like(q)
        pkg.pa_decode_weights(q, sv.kc, sv.vc, tables_of(sv.m, sv.names, sv.width), lens, sv.scale, out, sv.w, 1000, error_word=sv.err)
        sv.check(out.double().cpu().numpy(), hq)
        for s in range(B):
            _, w, _, tol = ref.attention(hq[s], sv.k[s], sv.v[s], sv.scale, sv.group)
            grow = np.zeros((Q + 1, sv.hkv))
            total[s] = np.concatenate([total[s], grow]) + w
            off[s] = np.concatenate([off[s], grow]) + tol + 2.0 ** -23 * total[s]
        target = torch.full((B, Q + 1, V), 1.0 / V, device="cuda")
        tokens = torch.from_numpy(sv.r.integers(0, V, (B, Q)).astype(np.int32)).cuda()
        u = torch.from_numpy((sv.r.random((B, Q + 1)) * 2 / V).astype(np.float32)).cuda()
        new, accepted = torch.zeros(B, Q + 1, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
        pkg.pa_verify_draft(target, None, tokens, u, new, accepted, context_lens=lens, lens_out=lens, error_word=sv.err)
        for s, n in enumerate(lens.tolist()):
            taken += len(sv.k[s]) - n
            assert sv.m.truncate(sv.names[s], n) is None
            sv.k[s], sv.v[s], total[s], off[s] = (x[:n] for x in (sv.k[s], sv.v[s], total[s], off[s]))
        pool = sv.w.cpu().numpy()
        for s in range(B):
            got = ref.slot_rows(pool, np.array(sv.m.block_table(sv.names[s])), len(total[s]), 16).astype(np.float64)
            assert (np.abs(got - total[s]) <= off[s]).all()
    assert taken > 0
    sv.done()
