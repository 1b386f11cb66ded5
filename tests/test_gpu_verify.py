"""pa_verify_draft against 64 bits: accepted numbers, drawn tokens, lengths."""
import numpy as np
import pytest
import torch

import cache_rows_reference as ref
import paged_kv_cache_29_gb300 as pkg
from paged_kv_cache_29_gb300 import _binding as pa

pytestmark = pytest.mark.gpu


def softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


class Verify:
    def __init__(self, B, Q, V, lookup=False, ragged=False, seed=0, spread=2.0, pad=0):
        r = np.random.default_rng(seed)
        logits = spread * r.standard_normal((B, Q + 1, V))
        self.target = softmax(logits)
        self.draft = None if lookup else softmax(logits[:, :Q] + 0.7 * r.standard_normal((B, Q, V)))
        pick = self.target[:, :Q] if lookup else self.draft
        run = np.cumsum(pick.astype(np.float64), -1)
        self.tokens = np.minimum((run <= r.random((B, Q, 1)) * run[..., -1:]).sum(-1), V - 1).astype(np.int32).reshape(B, Q)
        self.uniforms = r.random((B, Q + 1)).astype(np.float32)
        self.uniforms[self.uniforms >= 1] = 0.5
        self.count = r.integers(0, Q + 1, B).astype(np.int32) if ragged else None
        self.lens = r.integers(Q, 5000, B).astype(np.int32)
        self.pad = pad

    def run(self, in_place=False, **kw):
        def probs(x):
            if x is None:
                return None
            t = torch.full((*x.shape[:2], x.shape[2] + self.pad), float("nan"), device="cuda")
            t[..., :x.shape[2]] = torch.from_numpy(x)
            return t[..., :x.shape[2]]
        B, Q = self.tokens.shape
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((B, Q + 1), -9, dtype=torch.int32, device="cuda")
        accepted = torch.full((B,), -9, dtype=torch.int32, device="cuda")
        lens = torch.from_numpy(self.lens).cuda()
        lens_out = lens if in_place else torch.full_like(lens, -9)
        pkg.pa_verify_draft(probs(self.target), probs(self.draft), torch.from_numpy(self.tokens).cuda(), torch.from_numpy(self.uniforms).cuda(), out,
                           accepted, num_drafts=None if self.count is None else torch.from_numpy(self.count).cuda(), context_lens=lens,
                           lens_out=lens_out, error_word=self.err, **kw)
        return out.cpu().numpy(), accepted.cpu().numpy(), lens_out.cpu().numpy()

    def check(self, skip=(), **kw):
        out, accepted, lens = self.run(**kw)
        B, Q = self.tokens.shape
        seen = set()
        for s in range(B):
            if s in skip:
                assert (out[s] == -9).all() and accepted[s] == -9
                continue
            d = Q if self.count is None else int(self.count[s])
            a, token, near = ref.verify(self.target[s], None if self.draft is None else self.draft[s], self.tokens[s],
                                        self.uniforms[s].astype(np.float64), d)
            # Sums of 64 bits here, of 44 or more there: nearer borders say nothing.
            if near > 2.0 ** -43:
                assert accepted[s] == a and list(out[s]) == list(self.tokens[s][:a]) + [token] + [-1] * (Q - a), s
                assert lens[s] == self.lens[s] - (d - a)
            seen.add(a)
        return seen


@pytest.mark.parametrize("lookup", [False, True])
@pytest.mark.parametrize("B,Q,V", [(1, 4, 32000), (7, 1, 1), (5, 3, 2), (64, 5, 31), (33, 4, 1000), (16, 7, 1024), (9, 2, 1025), (3, 16, 50021),
                                   (150, 3, 4099), (400, 2, 777), (2, 64, 333), (20, 4, 131072), (6, 0, 5000), (1, 1, 1 << 20), (160, 1, 20011)])
def test_tokens(B, Q, V, lookup):
    Verify(B, Q, V, lookup, seed=B + Q + V).check()


@pytest.mark.parametrize("pad", [0, 1, 3, 64])
def test_ragged_and_padded_rows(pad):
    v = Verify(200, 6, 999, ragged=True, seed=pad, pad=pad)
    assert v.check() >= {0, 1, 2, 3}
    Verify(40, 6, 999, lookup=True, ragged=True, seed=pad, pad=pad).check(in_place=True)


def test_every_row_of_uniform_numbers_that_matters():
    """Uniform numbers of 0 and just below 1: the first and the last value of positive probability."""
    v = Verify(4, 2, 3000, seed=1)
    v.target[:, :, :5] = 0
    v.target[:, :, -7:] = 0
    v.target[:, :, [5, 2992]] = 1e-3
    v.draft[:] = v.target[:, :2]
    v.uniforms[:, :2] = 0.9999999
    v.tokens[:] = [100, 101]
    v.uniforms[:2, 2], v.uniforms[2:, 2] = 0.0, np.float32(1) - np.float32(2) ** -24
    out, accepted, _ = v.run()
    assert list(accepted) == [2, 2, 2, 2]              # equal distributions are always accepted
    assert list(out[:2, 2]) == [5, 5] and list(out[2:, 2]) == [2992, 2992]


def test_a_difference_that_leaves_nothing_falls_back_to_the_target():
    v = Verify(2, 1, 2000, seed=2)
    v.draft[:] = v.target[:, :1]
    v.target[:, 0, 7] = 0                              # x itself: p 0, and p <= q everywhere
    v.tokens[:] = 7
    assert v.check() == {0}


def test_tokens_of_no_probability_and_nan():
    v = Verify(4, 2, 500, seed=3)
    v.tokens[0] = [3, 4]
    v.target[0, 0, 3], v.draft[0, 0, 3] = 0.0, 0.0     # neither would draw it: rejected
    v.tokens[1] = [3, 4]
    v.draft[1, 0, 3] = 0.0                             # the draft would not: accepted
    v.target[2, :, 11] = np.nan                        # counts as 0
    v.draft[3, :, 12] = np.nan
    out, accepted, _ = v.run()
    assert accepted[0] == 0 and out[0, 0] != 3 and accepted[1] >= 1 and out[1, 0] == 3
    assert (out[2] != 11).all() and out[3, accepted[3]] >= 0


def test_flagged_sequences_are_left_out():
    v = Verify(8, 3, 600, ragged=True, seed=4)
    v.count[:] = 3
    v.tokens[1, 2], v.tokens[2, 0] = 600, -1           # outside the vocabulary
    v.count[3], v.count[4] = 4, -1
    v.tokens[5, 2], v.count[5] = 9999, 2               # not among the first d: unused
    v.target[6] = 0                                    # nothing to draw from
    v.check(skip=(1, 2, 3, 4, 6))
    assert int(v.err.item()) == pa.PA_DEVERR_TOKEN
    v = Verify(3, 3, 600, seed=5)
    v.uniforms[:, :3] = 0.99999
    v.target[:, 0, v.tokens[:, 0]] = 0
    v.lens[1] = 2
    v.check(skip=(1,))
    assert int(v.err.item()) == pa.PA_DEVERR_CONTEXT


def test_without_lengths_captured_and_replayed():
    v = Verify(5, 4, 3000, seed=6)
    t, d, x, u = (torch.from_numpy(a).cuda() for a in (v.target, v.draft, v.tokens, v.uniforms))
    out, acc = torch.zeros(5, 5, dtype=torch.int32, device="cuda"), torch.zeros(5, dtype=torch.int32, device="cuda")
    pkg.pa_verify_draft(t, d, x, u, out, acc)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.pa_verify_draft(t, d, x, u, out, acc)
    w = Verify(5, 4, 3000, seed=7)
    for a, b in ((t, w.target), (d, w.draft), (x, w.tokens), (u, w.uniforms)):
        a.copy_(torch.from_numpy(b))
    graph.replay()
    torch.cuda.synchronize()
    want = w.run()
    assert np.array_equal(out.cpu().numpy(), want[0]) and np.array_equal(acc.cpu().numpy(), want[1])


def test_drawn_tokens_are_distributed_as_the_targets():
    """Sequences of one distribution with random drafts and numbers: the first token's
    counts against its probabilities, within five standard deviations of each."""
    r = np.random.default_rng(8)
    B, V = 20000, 6
    p, q = np.float32([0.05, 0.4, 0.1, 0.25, 0.2, 0.0]), np.float32([0.3, 0.1, 0.1, 0.05, 0.2, 0.25])
    tokens = torch.from_numpy(r.choice(V, size=(B, 1), p=q / q.sum(dtype=np.float64)).astype(np.int32)).cuda()
    u = torch.from_numpy(r.random((B, 2), dtype=np.float32)).cuda()
    out, acc = torch.zeros(B, 2, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    target = torch.from_numpy(p).cuda().expand(B, 2, V)
    pkg.pa_verify_draft(target, torch.from_numpy(q).cuda().expand(B, 1, V), tokens, u, out, acc)
    counts = np.bincount(out[:, 0].cpu().numpy(), minlength=V)
    assert (np.abs(counts - B * p) <= 5 * np.sqrt(B * p * (1 - p))).all(), counts


@pytest.mark.parametrize("B", [1, 160])
def test_the_largest_vocabulary(B):
    """No drafts: draws from one row of 2^22 values, each sequence with its own number."""
    V = 1 << 22
    r = np.random.default_rng(9)
    p = softmax(2 * r.standard_normal(V))
    u = r.random((B, 1), dtype=np.float32)
    out, acc = torch.zeros(B, 1, dtype=torch.int32, device="cuda"), torch.ones(B, dtype=torch.int32, device="cuda")
    pkg.pa_verify_draft(torch.from_numpy(p).cuda().expand(B, 1, V), None, torch.zeros(B, 0, dtype=torch.int32, device="cuda"), torch.from_numpy(u).cuda(),
                       out, acc)
    run = np.cumsum(p.astype(np.float64))
    want = np.searchsorted(run, u[:, 0].astype(np.float64) * run[-1], side="right")
    assert np.array_equal(out[:, 0].cpu().numpy(), want) and not acc.any()
