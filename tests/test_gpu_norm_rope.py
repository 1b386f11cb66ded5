"""The norm and rotation calls on the GPU against 64 bits.

Bound of an output z = a cos - b sin (or b cos + a sin): half a step of its type
(2^-8 |z| for bf16, 2^-24 for fp32) plus 2^-20 (|a cos| + |b sin|). y = x r w is
off by at most 12 fp32 half-steps: the sum of up to 256 squares goes through 13
roundings, which count half in its root, the division, root, reciprocal and two
products add five, and each of z's two products and its sum one more: under
2^-24 * 16 = 2^-20."""
import numpy as np
import pytest
import torch

import rows_reference as ref
from paged_kv_cache_29_gb300 import _binding as pa
from test_gpu_int4 import bf16, dev, host, value

pytestmark = pytest.mark.gpu
MAX_POS = 300


def table(rot):
    half = rot // 2
    angle = np.arange(MAX_POS)[:, None] * 10000.0 ** (-np.arange(half) / half)
    return np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)


class Rows:
    """A fused projection's output, its parts, weights and positions."""

    def __init__(self, T, hq, hkv, d, dtype="bf16", rot=None, axes=1, seed=0, gain=1.0):
        rng = np.random.default_rng(seed)
        self.dtype, self.T, self.hq, self.hkv, self.d = dtype, T, hq, hkv, d
        x = rng.standard_normal((T, (hq + 2 * hkv) * d)) * gain
        w = 1 + 0.2 * rng.standard_normal((2, d))
        if dtype == "bf16":
            self.qkv, self.w = ref.bf16_value(bf16(x)), ref.bf16_value(bf16(w))
            self.dqkv, self.dw = dev(bf16(x)), dev(bf16(w))
        else:
            self.qkv, self.w = x.astype(np.float32), w.astype(np.float32)
            self.dqkv, self.dw = dev(self.qkv), dev(self.w)
        self.rot = d if rot is None else rot
        self.table = table(self.rot) if self.rot else None
        self.pos = rng.integers(0, MAX_POS, (axes, T)).astype(np.int32)
        self.axis = rng.integers(0, axes, self.rot // 2).tolist() if axes > 1 else None

    def parts(self, x):
        a, b = self.hq * self.d, (self.hq + self.hkv) * self.d
        cut = (x[:, :a], x[:, a:b], x[:, b:])
        return [c.reshape(self.T, -1, self.d) if isinstance(c, np.ndarray) else c.unflatten(1, (-1, self.d)) for c in cut]

    def out(self, heads):
        return torch.full((self.T, heads, self.d), 7.0, dtype=self.dqkv.dtype, device="cuda")

    def read(self, t):
        return value(host(t)) if self.dtype == "bf16" else t.cpu().numpy().astype(np.float64)

    def position_args(self):
        return (dev(self.pos) if self.rot else None), (dev(self.table) if self.rot else None)

    def want(self, which, **kw):
        x = self.parts(self.qkv)[which]
        w = kw.pop("weight", self.w[which])
        return ref.norm_rope(x, w, self.pos, self.table, pair_axis=self.axis, **kw)

    def check(self, got, which, rows=slice(None), **kw):
        want, size = self.want(which, **kw)
        half = 2.0 ** -8 if self.dtype == "bf16" else 2.0 ** -24
        over = np.abs(got - want)[rows] - (half * np.abs(want) + 2.0 ** -20 * size)[rows]
        assert over.size == 0 or over.max() <= 0, f"{over.max():.3g} over the bound"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,rot", [(16, 16), (64, 64), (80, 48), (96, 96), (128, 128), (128, 32), (128, 0), (192, 64), (256, 256)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope(dtype, d, rot, interleaved):
    r = Rows(37, 5, 2, d, dtype, rot, seed=d + rot)
    q, k, _ = r.parts(r.dqkv)
    pos, cs = r.position_args()
    q_out, k_out = r.out(5), r.out(2)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_norm_rope(q, k, pos, cs, q_out, k_out, r.dw[0], r.dw[1], interleaved=interleaved, error_word=err)
    assert int(err.item()) == 0
    r.check(r.read(q_out), 0, interleaved=interleaved)
    r.check(r.read(k_out), 1, interleaved=interleaved)


@pytest.mark.parametrize("axes", [2, 3, 4])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("sections", ["mixed", "blocks"])
def test_several_axes(axes, interleaved, sections):
    r = Rows(50, 4, 4, 128, axes=axes, seed=axes)
    if sections == "blocks":
        r.axis = sorted(i % axes for i in range(64))
    q, k, _ = r.parts(r.dqkv)
    q_out, k_out = r.out(4), r.out(4)
    pa.pa_norm_rope(q, k, *r.position_args(), q_out, k_out, r.dw[0], r.dw[1], interleaved=interleaved, pair_axis=r.axis)
    r.check(r.read(q_out), 0, interleaved=interleaved)
    r.check(r.read(k_out), 1, interleaved=interleaved)


def test_weights_offset_eps_and_no_norm():
    r = Rows(9, 4, 2, 64, seed=3)
    q, k, _ = r.parts(r.dqkv)
    q_out, k_out = r.out(4), r.out(2)
    pa.pa_norm_rope(q, k, *r.position_args(), q_out, k_out, r.dw[0], None, eps=0.3, weight_offset=1.0)
    r.check(r.read(q_out), 0, eps=0.3, weight_offset=1.0)
    r.check(r.read(k_out), 1, weight=None)
    w32 = torch.randn(64, device="cuda")
    pa.pa_norm_rope(q, k, *r.position_args(), q_out, k_out, None, w32)
    r.check(r.read(q_out), 0, weight=None)
    r.check(r.read(k_out), 1, weight=w32.cpu().numpy())


@pytest.mark.parametrize("gain", [0.0, 1e-15, 1e15])
def test_small_and_large_rows(gain):
    r = Rows(5, 3, 1, 128, seed=4, gain=gain)
    q, k, _ = r.parts(r.dqkv)
    q_out, k_out = r.out(3), r.out(1)
    pa.pa_norm_rope(q, k, *r.position_args(), q_out, k_out, r.dw[0], r.dw[1])
    r.check(r.read(q_out), 0)
    r.check(r.read(k_out), 1)


@pytest.mark.parametrize("T,hq,hkv", [(1, 1, 1), (1, 32, 8), (3, 64, 8), (2000, 4, 1), (700, 32, 32)])
def test_sizes_in_place(T, hq, hkv):
    """q and k of the projection turned where they are; v is left alone."""
    r = Rows(T, hq, hkv, 128, seed=T)
    q, k, v = r.parts(r.dqkv)
    before = v.clone()
    pa.pa_norm_rope(q, k, *r.position_args(), q, k, r.dw[0], r.dw[1])
    assert torch.equal(v, before)
    r.check(r.read(q.contiguous()), 0)
    r.check(r.read(k.contiguous()), 1)


def _slots(rng, T, nb, bs):
    slots = rng.permutation(nb * bs)[:T].astype(np.int64)
    if T > 6:
        slots[1], slots[5] = -1, nb * bs + 3
    return slots


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,bs", [(64, 16), (96, 5), (128, 16), (256, 1)])
@pytest.mark.parametrize("T", [1, 7, 90])
def test_append_writes_the_slots_and_nothing_else(dtype, d, bs, T):
    r = Rows(T, 4, 3, d, dtype, seed=d + T)
    nb = 100 // bs + 2
    slots = _slots(np.random.default_rng(T), T, nb, bs)
    q, k, v = r.parts(r.dqkv)
    kc = torch.full((nb, 3, bs, d), 7.0, dtype=r.dqkv.dtype, device="cuda")
    vc = kc.clone()
    q_out = r.out(4)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_norm_rope_append(q, k, v, *r.position_args(), dev(slots), q_out, kc, vc, r.dw[0], r.dw[1], error_word=err)
    assert int(err.item()) == (pa.PA_DEVERR_SLOT if T > 6 else 0)
    r.check(r.read(q_out), 0)
    ok = (slots >= 0) & (slots < nb * bs)
    flat = {n: r.read(c).transpose(0, 2, 1, 3).reshape(nb * bs, 3, d) for n, c in (("k", kc), ("v", vc))}
    got = np.zeros((T, 3, d))
    got[ok] = flat["k"][slots[ok]]
    r.check(got, 1, rows=ok)
    np.testing.assert_array_equal(flat["v"][slots[ok]], r.parts(r.qkv)[2][ok])
    untouched = np.setdiff1d(np.arange(nb * bs), slots[ok])
    assert (flat["k"][untouched] == 7.0).all() and (flat["v"][untouched] == 7.0).all()


def test_append_copies_v_bit_for_bit():
    """NaN payloads, infinities and subnormals of V arrive as they are."""
    r = Rows(4, 2, 2, 64, seed=8)
    bits = np.random.default_rng(8).integers(0, 1 << 16, (4, 2, 64)).astype(np.uint16)
    kc = torch.zeros(1, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    q, k, _ = r.parts(r.dqkv)
    pa.pa_norm_rope_append(q, k, dev(bits), *r.position_args(), dev(np.arange(4, dtype=np.int64)), r.out(2), kc, vc, r.dw[0], r.dw[1])
    np.testing.assert_array_equal(host(vc)[0, :, :4], bits.transpose(1, 0, 2))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 96, 128, 256])
@pytest.mark.parametrize("T", [1, 7, 90])
def test_append_int4_is_the_two_calls(dtype, d, T):
    r = Rows(T, 4, 3, d, dtype, seed=d + T)
    nb, bs = 12, 16
    slots = dev(_slots(np.random.default_rng(T), T, nb, bs))
    q, k, v = r.parts(r.dqkv)

    def pool():
        return [torch.full((nb, 3, bs, d // 2), 9, dtype=torch.uint8, device="cuda") for _ in range(2)] + \
            [torch.full((nb, 3, bs, 2), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    one, two = pool(), pool()
    q1, q2, k2 = r.out(4), r.out(4), r.out(3)
    pa.pa_norm_rope_append_int4(q, k, v, *r.position_args(), slots, q1, *one, r.dw[0], r.dw[1])
    pa.pa_norm_rope(q, k, *r.position_args(), q2, k2, r.dw[0], r.dw[1])
    pa.pa_reshape_and_cache_int4(k2, v.contiguous(), slots, *two)
    torch.cuda.synchronize()
    r.check(r.read(q1), 0)
    assert torch.equal(q1, q2)
    for a, b in zip(one, two):
        assert torch.equal(a, b)


def test_positions_outside_the_table_skip_their_tokens():
    r = Rows(20, 4, 2, 128, axes=3, seed=9)
    r.axis = [0] * 64                       # the other axes are checked all the same
    r.pos[0, 3], r.pos[1, 5], r.pos[2, 7] = -1, MAX_POS, 1 << 30
    bad = [3, 5, 7]
    q, k, v = r.parts(r.dqkv)
    q_out, k_out = r.out(4), r.out(2)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_norm_rope(q, k, *r.position_args(), q_out, k_out, r.dw[0], r.dw[1], pair_axis=r.axis, error_word=err)
    assert int(err.item()) == pa.PA_DEVERR_POSITION
    good = np.setdiff1d(np.arange(20), bad)
    assert (q_out[bad] == 7).all() and (k_out[bad] == 7).all()
    r.pos[:, bad] = 0
    r.check(r.read(q_out), 0, rows=good)
    r.check(r.read(k_out), 1, rows=good)
    kc = torch.full((2, 2, 16, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    r.pos[0, 3] = MAX_POS
    pa.pa_norm_rope_append(q, k, v, *r.position_args(), dev(np.arange(20, dtype=np.int64)), q_out, kc, vc, r.dw[0], r.dw[1],
                           pair_axis=r.axis)
    assert (kc[0, :, 3] == 7).all() and (vc[0, :, 3] == 7).all() and not (kc[0, :, 4] == 7).any()


def test_empty_call():
    r = Rows(0, 4, 2, 64, seed=1)
    q, k, _ = r.parts(r.dqkv)
    pa.pa_norm_rope(q, k, torch.zeros(0, dtype=torch.int32, device="cuda"), dev(r.table), q, k, r.dw[0], r.dw[1])


def test_steps_of_a_prompt_and_its_answer_over_a_4_bit_cache():
    """A prompt appended in two chunks, read back, then three decode steps of
    norm, rotation, quantising append and attention (one of them a captured
    graph), against 64 bits on the rows that the calls left in the pool."""
    hq, hkv, d, bs, nb = 8, 2, 128, 16, 12
    prompt = [70, 33]
    rng = np.random.default_rng(40)
    tables = rng.permutation(nb).astype(np.int32).reshape(2, 6)
    kc = torch.zeros(nb, hkv, bs, d // 2, dtype=torch.uint8, device="cuda")
    kp = torch.zeros(nb, hkv, bs, 2, dtype=torch.bfloat16, device="cuda")
    pool = [kc, kc.clone(), kp, kp.clone()]
    dt, err = dev(tables), torch.zeros(1, dtype=torch.int32, device="cuda")

    def slots(seq, row):
        return dev(tables[seq, row // bs].astype(np.int64) * bs + row % bs)

    wanted = [np.zeros((96, hkv, d)), np.zeros((96, hkv, d))]
    for lo, hi in ((0, 40), (40, 70)):
        seq = np.concatenate([np.full(max(0, min(n, hi) - lo), s) for s, n in enumerate(prompt)]).astype(int)
        row = np.concatenate([np.arange(lo, max(lo, min(n, hi))) for n in prompt]).astype(int)
        r = Rows(len(row), hq, hkv, d, seed=lo + 50)
        r.pos[0] = row
        q, k, v = r.parts(r.dqkv)
        pa.pa_norm_rope_append_int4(q, k, v, *r.position_args(), slots(seq, row), r.out(hq), *pool, r.dw[0], r.dw[1], error_word=err)
        kw = r.want(1)[0]
        for t in np.nonzero(seq == 0)[0]:
            wanted[0][row[t]] = kw[t]
    lens = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 70], device="cuda")
    k_all = torch.empty(103, hkv, d, dtype=torch.float32, device="cuda")
    v_all = torch.empty_like(k_all)
    pa.pa_gather_int4(*pool, dt, lens, starts, k_all, v_all, 96, error_word=err)
    step = ref.bf16_value(host(pool[2])[..., 1])
    off = np.abs(k_all[:70].cpu().numpy() - wanted[0][:70]).max()
    assert off <= step.max() / 2 + 2.0 ** -8 * np.abs(wanted[0]).max()     # half a step, and K's own rounding

    r = Rows(2, hq, hkv, d, seed=60)
    pos, cs = r.position_args()
    q, k, v = r.parts(r.dqkv)
    q_out, out = r.out(hq), r.out(hq)
    slot = torch.zeros(2, dtype=torch.int64, device="cuda")
    ws = torch.empty(pa.pa_decode_workspace_size_multi(2, 1, hq, d, 96), dtype=torch.uint8, device="cuda")

    def one_step():
        pa.pa_norm_rope_append_int4(q, k, v, pos, cs, slot, q_out, *pool, r.dw[0], r.dw[1], error_word=err)
        pa.pa_decode_int4(q_out, *pool, dt, lens, d ** -0.5, out, 96, workspace=ws, error_word=err)

    graph = None
    for i in range(3):
        fresh = Rows(2, hq, hkv, d, seed=61 + i)
        row = np.array(prompt) + i
        r.dqkv.copy_(fresh.dqkv)
        lens.copy_(dev((row + 1).astype(np.int32)))
        pos.copy_(dev(row[None].astype(np.int32)))
        slot.copy_(slots(np.arange(2), row))
        if i == 0:
            one_step()
        else:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    one_step()
            graph.replay()
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        fresh.pos[0] = row
        fresh.w = r.w
        fresh.check(fresh.read(q_out), 0)
        hp = [host(p) for p in pool]
        for s in range(2):
            codes, pairs = ref.quantise4(fresh.parts(fresh.qkv)[2][s])
            b, o = tables[s, row[s] // bs], row[s] % bs
            np.testing.assert_array_equal(hp[1][b, :, o], codes)
            np.testing.assert_array_equal(hp[3][b, :, o], pairs)
            want, tol = ref.attention4(fresh.read(q_out)[s][None], hp, tables[s], row[s] + 1, d ** -0.5, bs)
            assert (np.abs(fresh.read(out)[s] - want[0]) <= tol[0]).all()


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("lens", [[40] * 24, [40, 5000] * 12])
def test_calls_back_to_back_wait_for_one_another(lens, captured):
    """Attention and a rotation of its own q in place, in turn without a host
    wait: each call starts while the one before it still runs (the merge of
    sequences of one partition has nothing to do), and none may run ahead."""
    hq, hkv, d, bs, B = 8, 2, 128, 16, len(lens)
    width = 5000 // bs + 1
    g = torch.Generator("cuda").manual_seed(3)
    pool = [torch.randint(0, 256, (64, hkv, bs, d // 2), dtype=torch.uint8, device="cuda", generator=g) for _ in range(2)] + \
        [torch.rand(64, hkv, bs, 2, device="cuda", generator=g).sub(0.4).to(torch.bfloat16) for _ in range(2)]
    table = torch.randint(0, 64, (B, width), dtype=torch.int32, device="cuda", generator=g)
    n, rows, steps = dev(np.array(lens, np.int32)), Rows(B, hq, hkv, d, seed=70), 6
    pos, cs = rows.position_args()
    start, k, _ = (t.clone() for t in rows.parts(rows.dqkv))
    q, k_out = start.clone(), torch.empty_like(k)
    ws = torch.empty(pa.pa_decode_workspace_size_multi(B, 1, hq, d, 5000), dtype=torch.uint8, device="cuda")

    def run(outs, wait):
        for out in outs:
            pa.pa_decode_int4(q, *pool, table, n, d ** -0.5, out, 5000, workspace=ws)
            wait()
            pa.pa_norm_rope(q, k, pos, cs, q, k_out, rows.dw[0], rows.dw[1])
            wait()

    want = [torch.empty_like(q) for _ in range(steps)]
    run(want, torch.cuda.synchronize)
    got = [torch.empty_like(q) for _ in range(steps)]
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(got, lambda: None)
    for _ in range(3):
        q.copy_(start)
        graph.replay() if captured else run(got, lambda: None)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
