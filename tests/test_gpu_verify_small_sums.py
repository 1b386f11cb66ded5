"""pa_verify_draft where what is left to draw from is next to nothing: every sequence
that is not flagged gets its tokens, by the exact sums."""
import numpy as np
import pytest
import torch

import paged_kv_cache_29_gb300 as pkg

pytestmark = pytest.mark.gpu

TINY = 2.0 ** -149                                     # the least positive fp32 value


def uniforms():
    return np.float32([0.0, 2.0 ** -30, 0.25, 0.5, 0.5 + 2.0 ** -24, 0.75, 0.9, 1 - 2.0 ** -24])


def draw(target, draft, tokens, u, context_lens):
    B, Q = tokens.shape
    out = torch.full((B, Q + 1), -9, dtype=torch.int32, device="cuda")
    accepted = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    lens = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()
    pkg.pa_verify_draft(dev(target), dev(draft), dev(tokens), dev(u), out, accepted, context_lens=dev(context_lens), lens_out=lens,
                        error_word=err)
    assert int(err.item()) == 0
    return out.cpu().numpy(), accepted.cpu().numpy(), lens.cpu().numpy()


@pytest.mark.parametrize("V", [3, 700, 50021])
@pytest.mark.parametrize("unit", [1, 3, 1 << 22, 71362, 1 << 23, 1 << 30, 1 << 50])   # of the values, in 2^-149
@pytest.mark.parametrize("case", ["difference", "lookup", "target", "fallback"])
def test_next_to_nothing_is_drawn_from_exactly(V, unit, case):
    """difference: p - q of a rejected draft; lookup: p without the draft; target: all
    accepted; fallback: p <= q everywhere, p itself is drawn from."""
    r = np.random.default_rng(V + unit)
    u_last = uniforms()
    B = len(u_last)
    tail = np.unique(np.concatenate([[V - 1], r.integers(0, V, 5)]))
    tail = tail[tail != 1] if V > 3 else np.array([0, 2])
    p = np.zeros(V, np.float32)
    p[tail] = (r.integers(1, 5, len(tail)) * float(unit) * TINY).astype(np.float32)   # exact
    draft = None
    if case == "target":
        Q, x, target = 0, 0, p[None]
    else:
        Q, x, target = 1, 1, np.stack([p, np.full(V, 1 / V, np.float32)])              # p(x) = 0: rejected
        if case != "lookup":
            draft = np.zeros((1, V), np.float32)
            draft[0, x] = 0.5
            if case == "fallback":
                draft[0] += p
    rep = lambda a: None if a is None else np.repeat(a[None], B, 0)
    u = np.full((B, Q + 1), 0.5, np.float32)
    u[:, Q] = u_last
    lens = np.arange(100, 100 + B, dtype=np.int32)
    out, accepted, lens_out = draw(rep(target), rep(draft), np.full((B, Q), x, np.int32), u, lens)
    run = np.cumsum(p.astype(np.float64))              # multiples of 2^-149 by fewer than 53 bits: exact
    assert not accepted.any() and np.array_equal(lens_out, lens - Q)
    for s in range(B):
        want = int(np.argmax(run > float(u_last[s]) * run[-1]))
        assert list(out[s]) == [want] + [-1] * Q, (s, u_last[s])
