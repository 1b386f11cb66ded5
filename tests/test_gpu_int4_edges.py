"""4-bit decode at the edges of its values, against 64 bits: rows that are not
finite and are masked for some of the query tokens, value rows whose steps lie
far apart, queries and keys near the ends of bf16's range."""
import numpy as np
import pytest

import rows_reference as ref
from test_gpu_int4 import Batch, bf16, value

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


# --------------------------------------- steps of value rows that lie far apart


def attention4_weighted(q, pools, table, n, scale, block_size):
    """rows_reference.attention4 for one query token with a bound in which every row
    counts by its weight w:
      2^-8 |o|                      the rounding to bf16
      2^-11 sum w |s| c             each weight times s rounded to f16
      2^-25 max(w a) sum c          half of f16's smallest step, 2^-24, for products
                                    below f16's normal range: they are taken relative
                                    to the largest w a, a = |s| + 2^-12 |lo| of a row
      2 d sum w (|lo| + |s| c)      d as in attention4: errors of the weights themselves
    """
    _, hq, D = q.shape
    kc, vc, kp, vp = pools
    hkv = kc.shape[1]
    i = np.arange(n)
    blk, off = np.asarray(table)[i // block_size], i % block_size
    out, tol = np.zeros((hq, D)), np.zeros((hq, D))
    for qh in range(hq):
        h = qh // (hq // hkv)
        k = ref.values4(kc[blk, h, off], kp[blk, h, off])
        klo, ks = (ref.bf16_value(kp[blk, h, off][:, e]).astype(np.float64) for e in (0, 1))
        vlo, vs = (ref.bf16_value(vp[blk, h, off][:, e]).astype(np.float64) for e in (0, 1))
        code = ref.codes4(vc[blk, h, off]).astype(np.float64)
        x = q[0, qh]
        s = scale * (k @ x)
        w = np.exp(s - s.max())
        w /= w.sum()
        o = w @ (vlo[:, None] + vs[:, None] * code)
        size = abs(scale) * (np.abs(ks) * (ref.codes4(kc[blk, h, off]) @ np.abs(x)) + np.abs(klo) * np.abs(x).sum())
        d = size.max() * 2.0 ** -18 + 2.0 ** -20
        out[qh] = o
        tol[qh] = (2.0 ** -8 * np.abs(o) + 2.0 ** -11 * ((w * np.abs(vs)) @ code)
                   + 2.0 ** -25 * (w * (np.abs(vs) + 2.0 ** -12 * np.abs(vlo))).max() * code.sum(0)
                   + 2 * d * (w @ (np.abs(vlo)[:, None] + np.abs(vs)[:, None] * code)))
    return out, tol


def _row_weights(b, s, h):
    """Weights of sequence s's rows for the query heads of KV head h: [G][n]."""
    i = np.arange(b.lens[s])
    blk, off = b.table[s, i // b.bs], i % b.bs
    G = b.hq // b.hkv
    z = b.scale * value(b.q[s, 0, h * G:(h + 1) * G]) @ ref.values4(b.pools[0][blk, h, off], b.pools[2][blk, h, off]).T
    w = np.exp(z - z.max(-1, keepdims=True))
    return w / w.sum(-1, keepdims=True)


def _set_value_row(b, s, h, i, x):
    codes, pair = ref.quantise4(np.asarray(x, np.float32)[None])
    at = b.table[s, i // b.bs], h, i % b.bs
    b.pools[1][at], b.pools[3][at] = codes[0], pair[0]


def _check(b):
    got = b.upload().decode()[:, 0]
    assert int(b.err.item()) == 0
    for s, n in enumerate(b.lens):
        want, tol = attention4_weighted(value(b.q[s]), b.pools, b.table[s], n, b.scale, b.bs)
        worst = (np.abs(got[s] - want) - tol).max()
        assert worst <= 0, f"sequence {s} of {n} rows: {worst:.3g} over its bound"


SPREAD = [40, 100, 290, 700, 1500, 2300]


@pytest.mark.parametrize("group", [1, 4, 8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ratio", [16, 20, 24, 40, 60])
def test_a_row_of_no_weight_with_a_large_step(ratio, d, group):
    """The row of least weight has a step 2^ratio times the others': its share of
    the output is nothing, and the others keep their bits."""
    b = Batch(SPREAD, hq=2 * group, hkv=2, d=d, seed=ratio + group)
    b.scale *= 12
    rng = np.random.default_rng(ratio)
    for s in range(len(SPREAD)):
        for h in range(2):
            i = int(_row_weights(b, s, h).max(0).argmin())
            _set_value_row(b, s, h, i, rng.standard_normal(d) * 2.0 ** ratio)
    _check(b)


@pytest.mark.parametrize("ratio", [20, 40, 60])
def test_a_large_step_among_ordinary_weights(ratio):
    """Some rows with large steps and their ordinary share of the weight."""
    b = Batch(SPREAD, hq=8, hkv=2, seed=ratio)
    b.scale *= 4
    rng = np.random.default_rng(ratio)
    for s, n in enumerate(SPREAD):
        for i in rng.integers(0, n, 3):
            _set_value_row(b, s, 0, int(i), rng.standard_normal(128) * 2.0 ** ratio)
    _check(b)


@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("content", [0.0, 2.0 ** -30, 3.0, 1e6, 1e20])
def test_a_row_of_nearly_all_weight_and_one_value(content, where):
    """A row that takes nearly all the weight holds one value (a step of zero);
    where that is 0, the output is the others' small share."""
    b = Batch(SPREAD, hq=8, hkv=2, seed=77)
    G = b.hq // b.hkv
    for s, n in enumerate(SPREAD):
        i = {"first": 0, "middle": n // 2, "last": n - 1}[where]
        for h in range(2):
            b.q[s, 0, h * G:(h + 1) * G] = b.q[s, 0, h * G]
            x = value(b.q[s, 0, h * G])
            codes, pair = ref.quantise4((x * 2.2).astype(np.float32)[None])
            at = b.table[s, i // b.bs], h, i % b.bs
            b.pools[0][at], b.pools[2][at] = codes[0], pair[0]
            _set_value_row(b, s, h, i, np.full(128, content))
    _check(b)


@pytest.mark.parametrize("big", [12, 60])
@pytest.mark.parametrize("lead", [0, 10, 25, 37, 60])
def test_partitions_of_zero_rows_beside_one_of_large_steps(lead, big):
    """Zero value rows whose scores lead by `lead` (base 2) over those of a partition
    of large steps: parts of a sequence whose ranges differ by far join soundly."""
    b = Batch([2300, 700], hq=4, hkv=1, seed=lead + big)
    b.scale *= 0.01                                       # scores near 0
    b.q[:, :, :, 0] = bf16(np.float32(4.0))
    rng = np.random.default_rng(lead)
    for s, n in enumerate(b.lens):
        for i in range(n):
            at = b.table[s, i // b.bs], 0, i % b.bs
            large = i >= n - 60
            x = rng.standard_normal(128) * 0.01
            x[0] = 0.0 if large else lead * np.log(2.0) / (4.0 * b.scale)
            codes, pair = ref.quantise4(x.astype(np.float32)[None])
            b.pools[0][at], b.pools[2][at] = codes[0], pair[0]
            _set_value_row(b, s, 0, i, rng.standard_normal(128) * 2.0 ** big if large else np.zeros(128))
    _check(b)


@pytest.mark.parametrize("v_gain", [2.0 ** -98, 2.0 ** -60, 2.0 ** 60, 2.0 ** 98])
def test_steps_at_the_ends_of_the_range(v_gain):
    b = Batch(SPREAD, hq=8, hkv=2, seed=3, v_gain=v_gain)
    b.scale *= 4
    _check(b)


@pytest.mark.parametrize("group", [1, 8])
def test_steps_of_either_sign(group):
    """A row's value is lo + s c whatever the sign of s (the append writes none below 0)."""
    b = Batch(SPREAD, hq=2 * group, hkv=2, seed=61)
    b.scale *= 4
    flip = np.random.default_rng(62).random(b.pools[3].shape[:3])
    for pairs, below in ((b.pools[2], 0.3), (b.pools[3], 0.6)):
        pairs[..., 1] ^= np.where(flip < below, 0x8000, 0).astype(np.uint16)
    _check(b)


# ----------------------------------- queries and keys at the ends of the range


@pytest.mark.parametrize("gain", [-125, -110, 100, 112, 115, 120, 123])
def test_queries_of_any_size_with_ordinary_scores(gain):
    b = Batch([5, 600, 1500], hq=8, hkv=2, seed=9)
    b.q = bf16(np.clip(value(b.q), -3.9, 3.9) * 2.0 ** gain)
    b.scale *= 2.0 ** -gain
    b.upload()
    b.check(b.decode())


@pytest.mark.parametrize("gain", [1e-33, 1e33, 3e36])
def test_keys_of_any_size_with_ordinary_scores(gain):
    b = Batch([5, 600, 1500], hq=8, hkv=2, seed=19, k_gain=gain).upload()
    b.check(b.decode())


def test_zero_scale_weighs_rows_equally_whatever_the_keys():
    b = Batch([5, 600, 1500], hq=8, hkv=2, seed=20, k_gain=3e36)
    b.scale = 0.0
    b.upload()
    b.check(b.decode())


@pytest.mark.parametrize("group", [1, 8])
@pytest.mark.parametrize("power", [16, 20, 24])
def test_scores_up_to_2_to_the_27(power, group):
    """Scores of some 2^power to 5 * 2^power: where one row leads by more than the scores'
    error (2^-18 of their terms) it is the output. Below 2^27, 2^28 in base 2, the
    reference is off by half of fp32's step of 16 there at most, so that the f16
    operands, put at 2^7, stay between 2^-1 and 2^15.2."""
    b = Batch([5, 600, 1500], hq=2 * group, hkv=2, seed=power)
    b.scale *= 2.0 ** power
    got = b.upload().decode()[:, 0]
    assert np.isfinite(got).all()
    led = 0
    for s, n in enumerate(b.lens):
        i = np.arange(n)
        blk, off = b.table[s, i // b.bs], i % b.bs
        for qh in range(b.hq):
            h = qh // group
            x = value(b.q[s, 0, qh])
            z = b.scale * (ref.values4(b.pools[0][blk, h, off], b.pools[2][blk, h, off]) @ x)
            pair = ref.bf16_value(b.pools[2][blk, h, off]).astype(np.float64)
            size = b.scale * ((np.abs(pair[:, 0]) + 15 * pair[:, 1]) * np.abs(x).sum()).max()
            assert size < 2.0 ** 32 and np.abs(z).max() < 2.0 ** 27
            first, second = np.sort(z)[-1:-3:-1]
            if first - second > 2.0 ** -17 * size + 32:
                led += 1
                v = ref.values4(b.pools[1][blk, h, off], b.pools[3][blk, h, off])[z.argmax()]
                assert (np.abs(got[s, qh] - v) <= (2.0 ** -8 + 2.0 ** -10) * np.abs(v) + 2.0 ** -10 * np.abs(v).max()).all()
    assert led > b.hq
