"""Row weights are sums over the tokens that attend to a row: a token whose scores are not
finite does not reach the rows behind it."""
import numpy as np
import pytest
import torch

import cache_rows_reference as ref
from test_gpu_decode_rows import PLAIN, RING, Run, start_weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [s for s in RING + PLAIN if s[2] > 1], ids=str)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("long", [False, True])        # one partition each, and several
def test_a_token_that_is_not_finite_reaches_the_rows_that_it_sees(shape, bad, long):
    Q = shape[2]
    run = Run(shape, [Q, Q + 1, 40, 200, 512 - Q, 300] + [513, 1100] * long, seed=41)
    c = run.cache
    run.dq[:, 0] = bad                                 # the first token, every head
    start = start_weights(c)
    _, got = run.weights(start)
    for s, n in enumerate(run.lens):
        w, tol = np.zeros((n, run.hkv)), np.zeros((n, run.hkv))
        for j in range(1, Q):                          # the others, as calls of one token each
            see = n - Q + j + 1
            _, wj, _, tj = ref.attention(run.q[s, j:j + 1], c.k[s][:see], c.v[s][:see], run.scale, run.group)
            w[:see] += wj
            tol[:see] += tj
        g = ref.slot_rows(got, c.table[s], n, run.bs).astype(np.float64)
        behind = n - Q + 1                             # rows that the first token does not see
        off = np.abs(g[behind:] - w[behind:])
        assert (off <= tol[behind:] + 2.0 ** -24 * (w[behind:] + tol[behind:])).all(), (s, n)
        assert np.isnan(g[:behind]).all(), (s, n)
    assert int(run.err.item()) == 0
