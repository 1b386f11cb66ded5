"""4-bit decode at the edges of its values, against 64 bits: rows that are not
finite and are masked for some of the query tokens."""
import numpy as np
import pytest

import rows_reference as ref
from test_gpu_int4 import Batch, value

pytestmark = pytest.mark.gpu


# ------------------------------------- rows that only some query tokens see

POISON = {"nan": [0x7FC0, 0x7FC0], "inf": [0x7F80, 0x7F80], "minus inf, nan": [0xFF80, 0x7FC0], "finite lo": [0x3F80, 0x7F80],
          "finite step": [0x7F80, 0x3F80]}


@pytest.mark.parametrize("which", ["k", "v", "both"])
@pytest.mark.parametrize("poison", list(POISON))
@pytest.mark.parametrize("group,Q", [(1, 2), (4, 2), (2, 2), (1, 4), (1, 8), (2, 4)])
def test_a_bad_row_reaches_only_the_tokens_that_see_it(group, Q, poison, which):
    """The last row (a draft that may be rejected) is not finite: the tokens
    before the last are what they are without it."""
    lens = [Q, 16 + Q, 17, 40, 512, 1030, 1153, 2176]
    b = Batch(lens, hq=2 * group, hkv=2, Q=Q, seed=group + Q)
    for s, n in enumerate(lens):
        for pairs in b.pools[2:] if which == "both" else [b.pools[2 if which == "k" else 3]]:
            pairs[b.table[s, (n - 1) // b.bs], :, (n - 1) % b.bs] = POISON[poison]
    b.upload()
    with np.errstate(invalid="ignore"):
        for window in (0, 1, 20, 700):
            got = b.decode(window)
            assert poison != "nan" or np.isnan(got[:, Q - 1]).all()
            for s, n in enumerate(lens):
                want, tol = ref.attention4(value(b.q[s]), b.pools, b.table[s], n, b.scale, b.bs, window)
                assert (np.abs(got[s] - want) <= tol)[:Q - 1].all(), (s, window)
    assert int(b.err.item()) == 0


@pytest.mark.parametrize("Q,window", [(2, 5), (2, 64), (4, 17), (8, 33)])
def test_a_bad_row_that_has_left_the_later_tokens_windows(Q, window):
    """Row n - Q - window + 1 is seen by token 0 alone."""
    lens = [Q + window, 40 + window, 512 + window, 1100 + window]
    b = Batch(lens, hq=2, hkv=2, Q=Q, seed=Q + window)
    for s, n in enumerate(lens):
        i = n - Q - window + 1
        for pairs in b.pools[2:]:
            pairs[b.table[s, i // b.bs], :, i % b.bs] = POISON["nan"]
    got = b.upload().decode(window)
    assert np.isnan(got[:, 0]).all()
    with np.errstate(invalid="ignore"):
        for s, n in enumerate(lens):
            want, tol = ref.attention4(value(b.q[s]), b.pools, b.table[s], n, b.scale, b.bs, window)
            assert (np.abs(got[s] - want) <= tol)[1:].all(), s
