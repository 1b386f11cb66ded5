"""The cases that the 4-bit cache calls and the norm-and-rotation calls are
timed and compared on, with their plain forms.

Kinds of case:

  norm    per-head RMS norms of q and k and the position rotation, q and k read
          from one fused projection output ("dest": "out" writes q and k rows,
          "pool" writes q rows and appends K and V to a paged pool)
  cache   append a chunk of rows to a 4-bit cache, then read the whole
          context back as bf16 rows (a prompt processed in chunks)
  decode  decode attention over a 4-bit cache
  step    one layer's decode step over a 4-bit cache: norm, rotation and
          quantising append of the new rows, then attention

A 4-bit row (one token, one KV head) holds head_dim codes c in 0..15, two to a
byte (even dim in the low nibble), and a bf16 pair (lo, s): value = lo + s * c.
"""
import math
import random

import torch

own = False

MAX_POSITION = 32768


# ------------------------------------------------------------------- cases


def listed():
    return [
        # The tiny fp32 configuration: one token of one sequence. Latency.
        norm("norm one token fp32", tokens=1, heads=4, kv_heads=2, head_dim=64, dtype="f32", dest="out"),
        # One decode step of 128 sequences with grouped-query heads.
        norm("norm append decode batch", tokens=128, heads=32, kv_heads=8, head_dim=128, dest="pool"),
        # A prompt with images: three position axes, an odd number of tokens.
        norm("norm three axes prompt", tokens=4099, heads=32, kv_heads=8, head_dim=128, axes=3, dest="out"),
        # A long prompt appended at once, multi-head attention.
        norm("norm append long prompt", tokens=16384, heads=32, kv_heads=32, head_dim=128, dest="pool"),
        # The second chunk of one prompt.
        cache("cache4 one chunk", seqs=1, lens="same", low=1024, high=1024, chunk=512, kv_heads=8, head_dim=128),
        # The prompts of a whole batch, lengths spread like a serving batch's.
        cache("cache4 batch of prompts", seqs=128, lens="lognormal", low=16, high=8192, chunk=8192, kv_heads=8, head_dim=128),
        # One short sequence, the smallest attention call.
        decode("decode4 one short sequence", seqs=1, lens="same", low=17, high=17, heads=8, kv_heads=2, head_dim=64),
        # The serving batch: 128 sequences, grouped-query heads.
        decode("decode4 gqa batch", seqs=128, lens="lognormal", low=16, high=8192, heads=32, kv_heads=8, head_dim=128),
        # Multi-head attention, 32 sequences of 512 to 2,048 rows.
        decode("decode4 mha batch", seqs=32, lens="uniform", low=512, high=2048, heads=32, kv_heads=32, head_dim=128),
        # One very long sequence beside seven ordinary ones.
        decode("decode4 long skew", seqs=8, lens="skew", low=1500, high=100000, heads=32, kv_heads=8, head_dim=128),
        # Two draft tokens verified together in a local-attention layer.
        decode("decode4 two tokens window", seqs=128, lens="lognormal", low=16, high=8192, heads=32, kv_heads=8, head_dim=128, queries=2, window=1024),
        # One layer's decode step of the serving batch.
        step("step4 gqa batch", seqs=128, lens="lognormal", low=16, high=8192, heads=32, kv_heads=8, head_dim=128),
    ]


def norm(name, tokens, heads, kv_heads, head_dim, dtype="bf16", axes=1, rot_dim=None, interleaved=False, dest="out", block=16):
    return dict(name=name, kind="norm", tokens=tokens, heads=heads, kv_heads=kv_heads, head_dim=head_dim, dtype=dtype, axes=axes,
                rot_dim=rot_dim or head_dim, interleaved=interleaved, dest=dest, block=block)


def cache(name, seqs, lens, low, high, chunk, kv_heads, head_dim, block=16, lens_seed=1):
    return dict(name=name, kind="cache", seqs=seqs, lens=lens, low=low, high=high, chunk=chunk, kv_heads=kv_heads, head_dim=head_dim,
                block=block, lens_seed=lens_seed)


def decode(name, seqs, lens, low, high, heads, kv_heads, head_dim, queries=1, window=0, block=16, lens_seed=1):
    return dict(name=name, kind="decode", seqs=seqs, lens=lens, low=low, high=high, heads=heads, kv_heads=kv_heads, head_dim=head_dim,
                queries=queries, window=window, block=block, lens_seed=lens_seed)


def step(name, seqs, lens, low, high, heads, kv_heads, head_dim, block=16, lens_seed=1):
    return dict(decode(name, seqs, lens, low, high, heads, kv_heads, head_dim, block=block, lens_seed=lens_seed), kind="step",
                axes=1, rot_dim=head_dim, interleaved=False, dtype="bf16")


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["norm", "cache", "decode", "decode", "step"])
    head_dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 5])
    block = rng.choice([16, 16, 16, 32, 48])
    if kind == "norm":
        head_dim = rng.choice([64, 128, 128, 96, 256])
        heads = kv_heads * rng.choice([1, 2, 3, 4, 7, 8])
        most = 16384 * 96 * 128 // ((heads + 2 * kv_heads) * head_dim)
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        c = norm("", _log(rng, 1, min(16384, most) // (2 if dtype == "f32" else 1)), heads, kv_heads, head_dim, dtype=dtype,
                 axes=rng.choice([1, 1, 3]), rot_dim=rng.choice([head_dim, head_dim, head_dim // 2]), interleaved=rng.random() < 0.3,
                 dest=rng.choice(["out", "pool"]), block=block)
    else:
        lens = rng.choice(["uniform", "lognormal"])
        seqs = _log(rng, 1, 160)
        high = _log(rng, 1, 100000 // max(1, seqs // 16) // max(1, kv_heads // 8))
        low = max(0, min(high, rng.choice([0, 1, high // 4])))
        seed = rng.randrange(1 << 20)
        if kind == "cache":
            high = min(high, 8192)
            c = cache("", seqs, lens, min(low, high), high, _log(rng, 1, high), kv_heads, head_dim, block, seed)
        else:
            group = rng.choice([1, 2, 3, 4, 4, 5, 7, 8])
            high = min(high, 8192 if seqs > 8 else 100000)
            low = min(low, high)
            if kind == "decode":
                queries = rng.choice([1, 1, 1, min(2, 8 // group or 1)])
                c = decode("", seqs, lens, low, max(high, queries), group * kv_heads, kv_heads, head_dim, queries,
                           rng.choice([0, 0, _log(rng, 1, 2048)]), block, seed)
            else:
                high = min(max(high, 1), MAX_POSITION)
                c = step("", seqs, lens, min(max(low, 1), high), high, group * kv_heads, kv_heads, head_dim, block, seed)
    c.pop("name")
    return c


def _lens(c):
    """Rows of each sequence: set by the case alone."""
    rng = random.Random(c["lens_seed"])
    low, high, out = c["low"], c["high"], []
    for s in range(c["seqs"]):
        if c["lens"] == "same":
            n = high
        elif c["lens"] == "skew":
            n = high if s == 0 else low
        elif c["lens"] == "uniform":
            n = rng.randint(low, high)
        else:  # a prompt of mean 1,500 in a batch that allows 8,192 rows (lognormal, sigma 0.8), and an answer of up to 300
            mean = 1500 * high / 8192
            n = int(math.exp(rng.gauss(math.log(mean) - 0.32, 0.8))) + rng.randint(0, int(300 * high / 8192))
            n = min(high, max(low, n))
        q = c.get("queries", 1)
        out.append(n if n >= q or n == 0 else q)
    return out


def _seen(c, n):
    """Rows that the query tokens of a sequence of n rows attend to (their union), and the attended (query token, row) pairs."""
    q, w = c["queries"], c["window"] or n
    if n == 0:
        return 0, 0
    first = max(0, n - q + 1 - w)
    return n - first, sum(min(w, n - q + j + 1) for j in range(q))


def work(c):
    if c["kind"] == "norm":
        es = 2 if c["dtype"] == "bf16" else 4
        t, rows = c["tokens"], c["heads"] + c["kv_heads"]
        moved = rows + (c["kv_heads"] if c["dest"] == "pool" else 0)
        table = 4 * c["rot_dim"] * min(t, MAX_POSITION)
        return {"bytes": t * (2 * moved * c["head_dim"] * es + 4 * c["axes"] + (8 if c["dest"] == "pool" else 0)) + table,
                "flops": t * rows * c["head_dim"] * 7}
    row = c["head_dim"] // 2 + 4
    lens = _lens(c)
    if c["kind"] == "cache":
        new = sum(min(n, c["chunk"]) for n in lens)
        pair = 2 * c["kv_heads"]
        return {"bytes": pair * (new * (2 * c["head_dim"] + row) + sum(lens) * (row + 2 * c["head_dim"])) + 8 * new,
                "flops": pair * c["head_dim"] * (4 * new + 2 * sum(lens))}
    rows = sum(_seen(c, n)[0] for n in lens)
    pairs = sum(_seen(c, n)[1] for n in lens)
    q = c["seqs"] * c["queries"] * c["heads"] * c["head_dim"] * 2
    out = {"bytes": 2 * rows * c["kv_heads"] * row + 2 * q + 4 * sum(-(-n // c["block"]) for n in lens),
           "flops": 4 * pairs * c["heads"] * c["head_dim"]}
    if c["kind"] == "step":
        new = c["seqs"] * c["kv_heads"]
        out["bytes"] += q + 2 * new * (2 * c["head_dim"] + row) + c["seqs"] * (4 * c["rot_dim"] + 12)
        out["flops"] += c["seqs"] * (c["heads"] + c["kv_heads"]) * c["head_dim"] * 7
    return out


# ------------------------------------------------------------------ inputs


def _type(c):
    return torch.float32 if c.get("dtype") == "f32" else torch.bfloat16


def _pair_axis(c):
    """The position axis of each rotated pair: with three axes, time first, then height and width in equal shares."""
    pairs = c["rot_dim"] // 2
    if c["axes"] == 1:
        return [0] * pairs
    t = pairs // 4
    h = (pairs - t) // 2
    return [0] * t + [1] * h + [2] * (pairs - t - h)


def _table(c):
    """cos and sin of every position and pair, angles in 64 bits."""
    half = c["rot_dim"] // 2
    freq = 500000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    angle = torch.arange(MAX_POSITION, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()


def _projection(c, tokens, g):
    """A fused projection's output, its q, k and v parts, and the norms' weights."""
    dt, d = _type(c), c["head_dim"]
    cols = (c["heads"] + 2 * c["kv_heads"]) * d
    qkv = torch.randn(tokens, cols, device="cuda", generator=g).to(dt)
    a, b = c["heads"] * d, (c["heads"] + c["kv_heads"]) * d
    q = qkv[:, :a].unflatten(1, (c["heads"], d))
    k = qkv[:, a:b].unflatten(1, (c["kv_heads"], d))
    v = qkv[:, b:].unflatten(1, (c["kv_heads"], d))
    qw, kw = ((1 + 0.1 * torch.randn(d, device="cuda", generator=g)).to(dt) for _ in range(2))
    return dict(q=q, k=k, v=v, q_weight=qw, k_weight=kw, table=_table(c), pair_axis=_pair_axis(c),
                axis_index=torch.tensor(_pair_axis(c), device="cuda"), eps=1e-6, interleaved=c["interleaved"], rot=c["rot_dim"])


def _tables(c, lens, g):
    """Block tables over a pool that holds the sequences' blocks in random order, and the pool's size."""
    bs = c["block"]
    nblk = [-(-n // bs) for n in lens]
    total, width = max(1, sum(nblk)), max(1, max(nblk))
    perm = torch.randperm(total, device="cuda", generator=g).to(torch.int32)
    counts = torch.tensor(nblk, device="cuda")
    start = counts.cumsum(0) - counts
    col = torch.arange(width, device="cuda")
    idx = (start[:, None] + col).clamp(max=total - 1)
    tables = torch.where(col < counts[:, None], perm[idx], torch.full_like(perm[idx], -1))
    return tables.contiguous(), total


def _slots(tables, seq, row, bs):
    return tables[seq, row // bs].long() * bs + row % bs


def _flat_rows(lens, first):
    """(sequence, row) of every row from first[s] to lens[s], sequence by sequence."""
    n = torch.tensor([a - b for a, b in zip(lens, first)], device="cuda")
    seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), n)
    at = torch.arange(int(n.sum()), device="cuda") - torch.repeat_interleave(n.cumsum(0) - n, n)
    return seq, at + torch.tensor(first, device="cuda")[seq]


def _pool4(c, blocks, g):
    """A 4-bit pool of values near N(0, 1), K with a few stronger dims."""
    shape = (blocks, c["kv_heads"], c["block"], c["head_dim"])
    out = []
    for which in range(2):
        gain = torch.ones(c["head_dim"], device="cuda")
        if which == 0:
            gain[:: 17] = 2.0
        codes = torch.empty(*shape[:3], c["head_dim"] // 2, dtype=torch.uint8, device="cuda")
        params = torch.empty(*shape[:3], 2, dtype=torch.bfloat16, device="cuda")
        for a in range(0, blocks, 4096):
            b = min(blocks, a + 4096)
            x = torch.randn(b - a, *shape[1:], device="cuda", generator=g) * gain
            codes[a:b], params[a:b] = _quantise(x)
        out += [codes, params]
    return out[0], out[2], out[1], out[3]


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": c}
    if c["kind"] == "norm":
        t = c["tokens"]
        st |= _projection(c, t, g)
        if c["axes"] == 1:
            pos = torch.arange(t, device="cuda")[None] + torch.randint(0, MAX_POSITION - t, (1, 1), device="cuda", generator=g)
            if c["tokens"] <= 512:  # a decode batch: each token at its own sequence's end
                pos = torch.randint(0, MAX_POSITION, (1, t), device="cuda", generator=g)
        else:  # images of 32 x 32 patches one after another
            i = torch.arange(t, device="cuda")
            first = torch.randint(0, MAX_POSITION - t, (1,), device="cuda", generator=g)
            pos = torch.stack([first + i // 1024, first + i % 1024 // 32, first + i % 32])
        st["positions"] = pos.to(torch.int32).contiguous()
        st["q_out"] = torch.empty(t, c["heads"], c["head_dim"], dtype=_type(c), device="cuda")
        if c["dest"] == "out":
            st["k_out"] = torch.empty(t, c["kv_heads"], c["head_dim"], dtype=_type(c), device="cuda")
        else:
            bs = c["block"]
            blocks = -(-t // bs)
            st["slots"] = torch.randperm(blocks * bs, device="cuda", generator=g)[:t].contiguous()
            if t > 512:  # a prompt fills its blocks in order
                perm = torch.randperm(blocks, device="cuda", generator=g)
                i = torch.arange(t, device="cuda")
                st["slots"] = perm[i // bs] * bs + i % bs
            for n in ("k_cache", "v_cache"):
                st[n] = torch.zeros(blocks, c["kv_heads"], bs, c["head_dim"], dtype=_type(c), device="cuda")
        return st
    lens = _lens(c)
    st["max_len"] = max(lens)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["tables"], blocks = _tables(c, lens, g)
    st["k_cache"], st["v_cache"], st["k_params"], st["v_params"] = _pool4(c, blocks, g)
    st["scale"] = c["head_dim"] ** -0.5
    if c["kind"] == "cache":
        seq, row = _flat_rows(lens, [max(0, n - c["chunk"]) for n in lens])
        st["slots"] = _slots(st["tables"], seq, row, c["block"])
        for n in ("k_new", "v_new"):
            st[n] = torch.randn(len(seq), c["kv_heads"], c["head_dim"], device="cuda", generator=g).bfloat16()
        st["every"] = _flat_rows(lens, [0] * len(lens))
        starts = st["lens"].long()
        st["starts"] = (starts.cumsum(0) - starts).contiguous()
        for n in ("k_out", "v_out"):
            st[n] = torch.empty(sum(lens), c["kv_heads"], c["head_dim"], dtype=torch.bfloat16, device="cuda")
        return st
    shape = (c["seqs"], c["queries"], c["heads"], c["head_dim"])
    if c["kind"] == "decode":
        st["q"] = torch.randn(*shape, device="cuda", generator=g).bfloat16()
        if c["queries"] == 1:
            st["q"] = st["q"][:, 0].contiguous()
    else:
        st |= _projection(c, c["seqs"], g)
        st["positions"] = (st["lens"] - 1).clamp(min=0)[None].contiguous()
        st["slots"] = _slots(st["tables"], torch.arange(c["seqs"], device="cuda"), (st["lens"] - 1).long(), c["block"])
        st["q_out"] = torch.empty(c["seqs"], c["heads"], c["head_dim"], dtype=torch.bfloat16, device="cuda")
    st["out"] = torch.empty(shape if c["queries"] > 1 else (shape[0], *shape[2:]), dtype=torch.bfloat16, device="cuda")
    return st


# ------------------------------------------------------------- plain forms


def _bf16_toward(x, up):
    """fp32 values rounded to bf16 towards plus or minus infinity."""
    bits = x.view(torch.int32)
    cut = bits & -65536
    away = (cut != bits) & ((x > 0) if up else (x < 0))
    return torch.where(away, cut + 65536, cut).view(torch.float32)


def _quantise(x):
    """4-bit codes, two to a byte, and the (lo, s) pairs of rows x (fp32)."""
    lo = _bf16_toward(x.amin(-1, keepdim=True), up=False)
    s = _bf16_toward((x.amax(-1, keepdim=True) - lo) / torch.full_like(lo, 15), up=True)  # a quotient, no product with 1 / 15
    c = torch.where(s > 0, ((x - lo) / s).round().clamp(0, 15), torch.zeros_like(x)).to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4), torch.cat([lo, s], -1).bfloat16()


def _values(codes, params, dtype=torch.float32):
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(dtype)
    p = params.to(dtype)
    return p[..., 0:1] + p[..., 1:2] * c


def _norm_rotate(x, w, st):
    x = x.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + st["eps"]) * w.float()
    rot, half = st["rot"], st["rot"] // 2
    pos = st["positions"][st["axis_index"]].t().long()
    pair = torch.arange(half, device=x.device)
    cos = st["table"][pos, pair][:, None]
    sin = st["table"][pos, pair + half][:, None]
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if st["interleaved"] else (y[..., :half], y[..., half:rot])
    a, b = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([a, b], -1).flatten(-2) if st["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([r, y[..., rot:]], -1)


def _attend(q, st, c):
    """Attention of q over the rows that the tables give, padded to the longest sequence, fp32."""
    seqs, heads, kv, d, queries = c["seqs"], c["heads"], c["kv_heads"], c["head_dim"], c["queries"]
    n = st["lens"].long()[:, None]
    first = (n - queries + 1 - c["window"]).clamp(min=0) if c["window"] else torch.zeros_like(n)
    span = min(st["max_len"], c["window"] + queries - 1) if c["window"] else st["max_len"]
    row = first + torch.arange(span, device="cuda")
    block = st["tables"].gather(1, (row // c["block"]).clamp(max=st["tables"].shape[1] - 1)).clamp(min=0).long()
    at = row % c["block"]
    k = _values(st["k_cache"][block, :, at], st["k_params"][block, :, at])
    v = _values(st["v_cache"][block, :, at], st["v_params"][block, :, at])
    x = q.float().view(seqs, queries, kv, heads // kv, d).permute(0, 2, 1, 3, 4).reshape(seqs, kv, -1, d)
    score = (x @ k.permute(0, 2, 3, 1)).view(seqs, kv, queries, heads // kv, span) * st["scale"]
    last = n - queries + torch.arange(queries, device="cuda")
    sees = (row[:, None] <= last[..., None]) & ((row[:, None] > last[..., None] - c["window"]) if c["window"] else True)
    score = score.masked_fill(~sees[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = (score - top.masked_fill(top == -math.inf, 0)).exp()
    total = p.sum(-1, keepdim=True)
    p = (p / total.masked_fill(total == 0, 1)).view(seqs, kv, -1, span)
    o = (p @ v.permute(0, 2, 1, 3)).view(seqs, kv, queries, heads // kv, d).permute(0, 2, 1, 3, 4)
    return o.reshape(q.shape).to(q.dtype)


def _plain(st):
    c = st["case"]
    if c["kind"] == "norm":
        q, k = (_norm_rotate(st[n], st[n + "_weight"], st).to(_type(c)) for n in "qk")
        if c["dest"] == "out":
            return q, k
        block, at = st["slots"] // c["block"], st["slots"] % c["block"]
        st["k_cache"][block, :, at] = k
        st["v_cache"][block, :, at] = st["v"]
        return q, st["k_cache"], st["v_cache"]
    if c["kind"] == "cache":
        _append4(st, st["k_new"].float(), st["v_new"].float())
        seq, row = st["every"]
        block, at = st["tables"][seq, row // c["block"]].long(), row % c["block"]
        return tuple(_values(st[n + "_cache"][block, :, at], st[n + "_params"][block, :, at]).bfloat16() for n in "kv")
    if c["kind"] == "decode":
        return _attend(st["q"], st, c)
    q, k = (_norm_rotate(st[n], st[n + "_weight"], st).bfloat16() for n in "qk")
    _append4(st, k.float(), st["v"].float())
    return q, _attend(q, st, c)


def _append4(st, k, v):
    bs = st["case"]["block"]
    block, at = st["slots"] // bs, st["slots"] % bs
    st["k_cache"][block, :, at], st["k_params"][block, :, at] = _quantise(k)
    st["v_cache"][block, :, at], st["v_params"][block, :, at] = _quantise(v)


# ------------------------------------------------------ the framework's calls


def run(st):
    if not own:
        return _plain(st)
    import paged_kv_cache_29_gb300 as pa
    c = st["case"]
    if c["kind"] in ("norm", "step"):
        options = dict(q_weight=st["q_weight"], k_weight=st["k_weight"], eps=st["eps"], interleaved=st["interleaved"],
                       pair_axis=st["pair_axis"] if c["axes"] > 1 else None)
    if c["kind"] == "norm":
        if c["dest"] == "out":
            pa.pa_norm_rope(st["q"], st["k"], st["positions"], st["table"], st["q_out"], st["k_out"], **options)
            return st["q_out"], st["k_out"]
        pa.pa_norm_rope_append(st["q"], st["k"], st["v"], st["positions"], st["table"], st["slots"], st["q_out"], st["k_cache"],
                               st["v_cache"], **options)
        return st["q_out"], st["k_cache"], st["v_cache"]
    pool = [st[n] for n in ("k_cache", "v_cache", "k_params", "v_params")]
    if c["kind"] == "cache":
        pa.pa_reshape_and_cache_int4(st["k_new"], st["v_new"], st["slots"], *pool)
        pa.pa_gather_int4(*pool, st["tables"], st["lens"], st["starts"], st["k_out"], st["v_out"], st["max_len"])
        return st["k_out"], st["v_out"]
    if c["kind"] == "step":
        pa.pa_norm_rope_append_int4(st["q"], st["k"], st["v"], st["positions"], st["table"], st["slots"], st["q_out"], *pool, **options)
    q = st["q_out"] if c["kind"] == "step" else st["q"]
    if "workspace" not in st:  # scratch that a program keeps beside its pool
        need = pa.pa_decode_workspace_size_multi(c["seqs"], c["queries"], c["heads"], c["head_dim"], st["max_len"])
        st["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    pa.pa_decode_int4(q, *pool, st["tables"], st["lens"], st["scale"], st["out"], st["max_len"], window=c["window"],
                      workspace=st["workspace"])
    return (q, st["out"]) if c["kind"] == "step" else st["out"]


# --------------------------------------------------------------- 64 bits


def _exact_norm(x, w, st):
    """Norm and rotation in 64 bits, as a product with each pair's rotation written out."""
    x = x.double()
    y = x / ((x.square().sum(-1, keepdim=True) / x.shape[-1] + st["eps"]).sqrt()) * w.double()
    rot, half = st["rot"], st["rot"] // 2
    out = y.clone()
    for i in range(half):
        rowi = st["positions"][st["pair_axis"][i]].long()
        cos, sin = (st["table"][rowi, i + o].double()[:, None] for o in (0, half))
        a, b = (2 * i, 2 * i + 1) if st["interleaved"] else (i, i + half)
        out[..., a] = y[..., a] * cos - y[..., b] * sin
        out[..., b] = y[..., b] * cos + y[..., a] * sin
    return out


def _exact_cache(x):
    """What a 4-bit row stands for, in 64 bits but for the pair (lo, s), which is held in bf16."""
    x = x.double()
    lo = _bf16_toward(x.amin(-1, keepdim=True).float(), up=False).double()
    s = _bf16_toward(((x.amax(-1, keepdim=True) - lo) / 15).float(), up=True).double()
    return lo + s * ((x - lo) / s.clamp(min=1e-300)).round().clamp(0, 15)


def _exact_rows(st, c, s, n):
    """K and V of sequence s in 64 bits, [kv_heads][n][head_dim]."""
    blocks = st["tables"][s, : -(-n // c["block"])].long()
    got = []
    for which in "kv":
        x = _values(st[which + "_cache"][blocks], st[which + "_params"][blocks], torch.float64)
        got.append(x.transpose(0, 1).flatten(1, 2)[:, :n])
    return got


def _exact_attention(q, st, c, new=None):
    out = torch.zeros(c["seqs"], c["queries"], c["heads"], c["head_dim"], dtype=torch.float64, device="cuda")
    q = q.double().view(out.shape)
    group = c["heads"] // c["kv_heads"]
    for s, n in enumerate(_lens(c)):
        if n == 0:
            continue
        k, v = _exact_rows(st, c, s, n)
        if new is not None:
            k[:, n - 1], v[:, n - 1] = new[0][s], new[1][s]
        for j in range(c["queries"]):
            end = n - c["queries"] + j + 1
            start = max(0, end - c["window"]) if c["window"] else 0
            x = q[s, j].view(c["kv_heads"], group, -1)
            w = torch.softmax(torch.einsum("hgd,hnd->hgn", x, k[:, start:end]) * st["scale"], -1)
            out[s, j] = torch.einsum("hgn,hnd->hgd", w, v[:, start:end]).reshape(c["heads"], -1)
    return out


def exact(c, seed):
    st = prepare(c, seed)
    if c["kind"] == "norm":
        q, k = (_exact_norm(st[n], st[n + "_weight"], st) for n in "qk")
        if c["dest"] == "out":
            return q, k
        pools = []
        for x in (k, st["v"].double()):
            flat = torch.zeros(st["k_cache"].shape[0] * c["block"], c["kv_heads"], c["head_dim"], dtype=torch.float64, device="cuda")
            flat[st["slots"]] = x
            pools.append(flat.unflatten(0, (-1, c["block"])).transpose(1, 2).contiguous())
        return q, *pools
    if c["kind"] == "cache":
        lens, outs = _lens(c), []
        new = [max(0, n - c["chunk"]) for n in lens]
        for which in "kv":
            rows = _exact_cache(st[which + "_new"])
            parts, at = [], 0
            for s, n in enumerate(lens):
                blocks = st["tables"][s, : -(-n // c["block"])].long()
                old = _values(st[which + "_cache"][blocks], st[which + "_params"][blocks], torch.float64)
                old = old.transpose(1, 2).flatten(0, 1)[: new[s]]
                parts += [old, rows[at: at + n - new[s]]]
                at += n - new[s]
            outs.append(torch.cat(parts))
        return tuple(outs)
    if c["kind"] == "decode":
        return _exact_attention(st["q"], st, c).view(st["out"].shape)
    q, k = (_exact_norm(st[n], st[n + "_weight"], st).bfloat16() for n in "qk")
    out = _exact_attention(q, st, c, (_exact_cache(k), _exact_cache(st["v"])))
    return _exact_norm(st["q"], st["q_weight"], st), out.view(st["out"].shape)
