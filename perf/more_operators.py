"""The cases that the calls which choose a cache's rows are timed and compared
on, with their plain forms.

Kinds of case:

  sinks    decode attention of each sequence's last tokens over a sliding window
           and the sequence's first rows, which stay visible
  weights  decode attention that adds every row's attention weight, summed over
           the query heads of its KV head, to an accumulator beside the cache
  evict    for each sequence and KV head the rows with the largest accumulated
           weights stay (and the first and the last ones); they move together,
           in place or into other blocks
  verify   drafted tokens are accepted or rejected against the target's
           probabilities, and one more token is drawn, from given random numbers

Pools are [block][kv_head][block_size][head_dim]; row i of a sequence is row
i % block_size of block table[i // block_size].
"""
import math
import random

import torch

own = False

# ------------------------------------------------------------------- cases


def listed():
    return [
        # One short sequence of an fp32 model, window and sinks smaller than it. Latency.
        sinks("sinks one short sequence", seqs=1, lens="same", low=40, high=40, heads=8, kv_heads=2, head_dim=64, window=16, first=4, dtype="f32"),
        # The serving batch in a layer with a window of 1,024: endless generation.
        sinks("sinks gqa batch", seqs=128, lens="lognormal", low=16, high=8192, heads=32, kv_heads=8, head_dim=128, window=1024, first=4),
        # Two draft tokens, one very long sequence beside seven ordinary ones.
        sinks("sinks drafts long skew", seqs=8, lens="skew", low=1500, high=100000, heads=32, kv_heads=8, head_dim=128, window=16384, first=64, queries=2),
        # The smallest call: one sequence of 17 rows.
        weights("weights one short sequence", seqs=1, lens="same", low=17, high=17, heads=8, kv_heads=2, head_dim=64),
        # The serving batch: 128 sequences, grouped-query heads.
        weights("weights gqa batch", seqs=128, lens="lognormal", low=16, high=8192, heads=32, kv_heads=8, head_dim=128),
        # One very long sequence beside seven ordinary ones.
        weights("weights long skew", seqs=8, lens="skew", low=1500, high=100000, heads=32, kv_heads=8, head_dim=128),
        # One sequence some blocks over its budget, into blocks of its own (its prompt's are shared).
        evict("evict one sequence", seqs=1, lens="same", low=600, high=600, share=0.85, kv_heads=8, head_dim=128, first=4, last=64, place="other"),
        # The serving batch cut to half of its rows, in place.
        evict("evict gqa batch", seqs=128, lens="lognormal", low=16, high=8192, share=0.5, kv_heads=8, head_dim=128, first=4, last=128, place="same"),
        # Prompts just read, one of 100,000 rows, to a quarter; 8-bit rows with a scale each.
        evict("evict long skew int8", seqs=8, lens="skew", low=1500, high=100000, share=0.25, kv_heads=8, head_dim=128, first=16, last=256, dtype="int8", place="other"),
        # One conversation, four draft tokens.
        verify("verify one sequence", seqs=1, drafts=4, vocab=32000),
        # Drafts by prompt lookup (no probabilities of their own), a ragged batch, an odd vocabulary.
        verify("verify lookup ragged", seqs=37, drafts=7, vocab=50021, draft="lookup", ragged=True),
        # The serving batch, four draft tokens from a small model, a large vocabulary.
        verify("verify batch", seqs=128, drafts=4, vocab=131072),
    ]


def sinks(name, seqs, lens, low, high, heads, kv_heads, head_dim, window, first, queries=1, dtype="bf16", block=16, lens_seed=1):
    return dict(name=name, kind="sinks", seqs=seqs, lens=lens, low=low, high=high, heads=heads, kv_heads=kv_heads, head_dim=head_dim,
                window=window, first=first, queries=queries, dtype=dtype, block=block, lens_seed=lens_seed)


def weights(name, seqs, lens, low, high, heads, kv_heads, head_dim, queries=1, dtype="bf16", block=16, lens_seed=1):
    return dict(name=name, kind="weights", seqs=seqs, lens=lens, low=low, high=high, heads=heads, kv_heads=kv_heads, head_dim=head_dim,
                window=0, first=0, queries=queries, dtype=dtype, block=block, lens_seed=lens_seed)


def evict(name, seqs, lens, low, high, share, kv_heads, head_dim, first, last, dtype="bf16", place="same", block=16, lens_seed=1):
    return dict(name=name, kind="evict", seqs=seqs, lens=lens, low=low, high=high, share=share, kv_heads=kv_heads, head_dim=head_dim,
                first=first, last=last, dtype=dtype, place=place, block=block, lens_seed=lens_seed)


def verify(name, seqs, drafts, vocab, draft="model", ragged=False, lens_seed=1):
    return dict(name=name, kind="verify", seqs=seqs, drafts=drafts, vocab=vocab, draft=draft, ragged=ragged, lens_seed=lens_seed)


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["sinks", "weights", "evict", "verify"])
    seed = rng.randrange(1 << 20)
    if kind == "verify":
        drafts, vocab = rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 11, 16]), _log(rng, 1000, 200000)
        seqs = _log(rng, 1, min(256, 128 * 9 * 131072 // ((2 * drafts + 1) * vocab)))
        c = verify("", seqs, drafts, vocab, rng.choice(["model", "model", "lookup"]), rng.random() < 0.4, seed)
    else:
        head_dim, kv_heads, block = rng.choice([64, 128, 128]), rng.choice([1, 2, 4, 8, 8, 5]), rng.choice([16, 16, 16, 32, 48])
        seqs, lens = _log(rng, 1, 160), rng.choice(["uniform", "lognormal"])
        high = _log(rng, 1, 100000 // max(1, seqs // 16) // max(1, kv_heads // 8))
        high = min(high, 8192 if seqs > 8 else 100000)
        low = max(0, min(high, rng.choice([0, 1, high // 4])))
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if dtype == "f32":
            high = max(1, high // 2)
        low = min(low, high)
        if kind == "evict":
            c = evict("", seqs, lens, low, high, rng.choice([0.25, 0.5, 0.8, rng.uniform(0.05, 1)]), kv_heads, head_dim,
                      rng.choice([0, 1, 4, 64]), rng.choice([0, 1, 32, 300]), rng.choice([dtype, "int8", "int4"]), rng.choice(["same", "other"]), block, seed)
        else:
            group = rng.choice([1, 2, 3, 4, 4, 5, 7, 8])
            queries = rng.choice([1, 1, 1, min(2, 8 // group or 1)]) if dtype == "bf16" else 1
            high = max(high, queries)
            if kind == "weights":
                c = weights("", seqs, lens, low, high, group * kv_heads, kv_heads, head_dim, queries, dtype, block, seed)
            else:
                c = sinks("", seqs, lens, low, high, group * kv_heads, kv_heads, head_dim, _log(rng, 1, 16384), rng.choice([0, 1, 4, 16, 100]), queries,
                          dtype, block, seed)
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


def _keep(c, n):
    """Rows that a sequence of n rows keeps: its share, and at least the first and last ones."""
    return min(n, max(int(round(n * c["share"])), c["first"] + c["last"]))


def _row_bytes(c):
    """Bytes of a row of K (or V) and KV head, and of what stands beside it for 8- and 4-bit rows."""
    d = c["head_dim"]
    return {"f32": (4 * d, 0), "bf16": (2 * d, 0), "int8": (d, 4), "int4": (d // 2, 4)}[c["dtype"]]


def _seen(c, n):
    """Rows that the query tokens of a sequence of n rows attend to (their union), and the attended (query token, row) pairs."""
    q, w, f = c["queries"], c["window"] or n, c["first"]
    if n == 0:
        return 0, 0
    start = max(0, n - q + 1 - w)
    rows = n - start + min(start, f)
    pairs = 0
    for j in range(q):
        last = n - q + j
        begin = max(0, last + 1 - w)
        pairs += last + 1 - begin + min(begin, f)
    return rows, pairs


def work(c):
    if c["kind"] == "verify":
        # One row of the target's probabilities for each sequence, and the draft's where a token was rejected: the
        # inputs accept a token with probability 0.7 (drafts of a model; a looked-up token is accepted with its own).
        rows = c["seqs"] * (2 - 0.7 ** c["drafts"] if c["draft"] == "model" else 1)
        return {"bytes": int(rows * 4 * c["vocab"]) + c["seqs"] * (16 * c["drafts"] + 16), "flops": int(2 * rows * c["vocab"])}
    lens = _lens(c)
    if c["kind"] == "evict":
        row, extra = _row_bytes(c)
        moved = 0
        for n in lens:  # rows behind the first that goes, by its expected place (all of them into other blocks)
            k = _keep(c, n)
            free = n - min(n, c["first"] + c["last"])
            moved += k if c["place"] == "other" else 0 if k == n else max(0, k - c["first"] - free // (n - k + 1))
        return {"bytes": c["kv_heads"] * (4 * sum(lens) + moved * 2 * (2 * (row + extra) + 4)) + 12 * c["seqs"], "flops": c["kv_heads"] * sum(lens)}
    es = 4 if c["dtype"] == "f32" else 2
    rows = sum(_seen(c, n)[0] for n in lens)
    pairs = sum(_seen(c, n)[1] for n in lens)
    q = c["seqs"] * c["queries"] * c["heads"] * c["head_dim"] * es
    out = {"bytes": 2 * rows * c["kv_heads"] * c["head_dim"] * es + 2 * q + 4 * sum(-(-n // c["block"]) for n in lens),
           "flops": 4 * pairs * c["heads"] * c["head_dim"]}
    if c["kind"] == "weights":
        out["bytes"] += 8 * rows * c["kv_heads"]
        out["flops"] += 2 * pairs * c["heads"]
    return out


# ------------------------------------------------------------------ inputs


def _tables(c, lens, g, spare=0):
    """Block tables over a pool that holds the sequences' blocks in random order, and how many blocks they take."""
    bs = c["block"]
    nblk = [-(-n // bs) for n in lens]
    total, width = max(1, sum(nblk)), max(1, max(nblk))
    perm = torch.randperm(total, device="cuda", generator=g).to(torch.int32) + spare
    counts = torch.tensor(nblk, device="cuda")
    start = counts.cumsum(0) - counts
    col = torch.arange(width, device="cuda")
    idx = (start[:, None] + col).clamp(max=total - 1)
    tables = torch.where(col < counts[:, None], perm[idx], torch.full_like(perm[idx], -1))
    return tables.contiguous(), total


def _verify_inputs(c, g, st):
    b, q, v = c["seqs"], c["drafts"], c["vocab"]
    logits = 2.5 * torch.randn(b, q + 1, v, device="cuda", generator=g)
    st["target"] = logits.softmax(-1)
    if c["draft"] == "model":
        # The draft's logits are the target's with noise of 0.77: the two overlap by 0.7.
        st["draft"] = (logits[:, :q] + 0.77 * torch.randn(b, q, v, device="cuda", generator=g)).softmax(-1)
        pick = st["draft"]
    else:
        st["draft"] = None
        pick = st["target"][:, :q].square()
    at = pick.double().cumsum(-1)
    u = torch.rand(b, q, 1, device="cuda", generator=g, dtype=torch.float64)
    st["tokens"] = (at <= u * at[..., -1:]).sum(-1).clamp(max=v - 1).to(torch.int32)
    st["uniforms"] = torch.rand(b, q + 1, device="cuda", generator=g)
    st["num_drafts"] = torch.randint(0, q + 1, (b,), device="cuda", generator=g).to(torch.int32) if c["ragged"] else None
    st["lens"] = torch.randint(q + 1, 8192, (b,), device="cuda", generator=g).to(torch.int32)
    st["lens_out"] = torch.empty_like(st["lens"])
    st["out_tokens"] = torch.empty(b, q + 1, dtype=torch.int32, device="cuda")
    st["accepted"] = torch.empty(b, dtype=torch.int32, device="cuda")
    return st


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": c}
    if c["kind"] == "verify":
        return _verify_inputs(c, g, st)
    lens = _lens(c)
    st["max_len"] = max(lens)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["tables"], blocks = _tables(c, lens, g)
    d, bs, kv = c["head_dim"], c["block"], c["kv_heads"]
    if c["kind"] == "evict":
        keep = [_keep(c, n) for n in lens]
        st["keep"] = torch.tensor(keep, dtype=torch.int32, device="cuda")
        st["lens_out"] = torch.empty_like(st["lens"])
        st["tables_out"] = st["tables"]
        if c["place"] == "other":
            st["tables_out"], more = _tables(c, keep, g, spare=blocks)
            blocks += more
            width = st["tables"].shape[1]
            st["tables_out"] = torch.nn.functional.pad(st["tables_out"], (0, width - st["tables_out"].shape[1]), value=-1).contiguous()
    shape = (blocks, kv, bs, d)
    if c["dtype"] in ("bf16", "f32"):
        st["k_cache"], st["v_cache"] = (torch.randn(*shape, device="cuda", generator=g).to(torch.float32 if c["dtype"] == "f32" else torch.bfloat16)
                                        for _ in range(2))
    elif c["dtype"] == "int8":
        st["k_cache"], st["v_cache"] = (torch.randint(-127, 128, shape, device="cuda", generator=g, dtype=torch.int8) for _ in range(2))
        st["k_params"], st["v_params"] = (torch.rand(*shape[:3], device="cuda", generator=g) for _ in range(2))
    else:
        st["k_cache"], st["v_cache"] = (torch.randint(0, 256, (*shape[:3], d // 2), device="cuda", generator=g, dtype=torch.uint8) for _ in range(2))
        st["k_params"], st["v_params"] = (torch.randn(*shape[:3], 2, device="cuda", generator=g).bfloat16() for _ in range(2))
    # Accumulated weights: a few rows that many tokens looked at, most hardly at all.
    saved = (2 * torch.randn(*shape[:3], device="cuda", generator=g) - 3).exp()
    st["row_weights"] = saved.clone()
    if c["kind"] == "evict":
        if c["place"] == "same":
            st["saved"] = saved
        return st
    dt = st["k_cache"].dtype
    q_shape = (c["seqs"], c["queries"], c["heads"], d) if c["queries"] > 1 else (c["seqs"], c["heads"], d)
    st["q"] = torch.randn(*q_shape, device="cuda", generator=g).to(dt)
    if c["kind"] == "weights":
        st["q"] = (1.5 * st["q"].float()).to(dt)  # scores wide enough that some rows matter
    st["out"] = torch.empty_like(st["q"])
    st["scale"] = d ** -0.5
    return st


# ------------------------------------------------------------- plain forms


def _attend(st, c):
    """Attention over the rows that each query token sees, fp32: the output, and the weights with the rows they belong to."""
    seqs, heads, kv, d, queries, bs = c["seqs"], c["heads"], c["kv_heads"], c["head_dim"], c["queries"], c["block"]
    n = st["lens"].long()[:, None]
    if c["window"]:
        start = (n - queries + 1 - c["window"]).clamp(min=0)
        span = min(st["max_len"], c["window"] + queries - 1)
        first = torch.arange(min(c["first"], st["max_len"]), device="cuda").expand(seqs, -1)
        row = torch.cat([first, start + torch.arange(span, device="cuda")], 1)
        own_place = torch.cat([first < start, torch.ones(seqs, span, dtype=torch.bool, device="cuda")], 1)  # a first row inside the window counts there
    else:
        row = torch.arange(st["max_len"], device="cuda").expand(seqs, -1)
        own_place = torch.ones_like(row, dtype=torch.bool)
    block = st["tables"].gather(1, (row // bs).clamp(max=st["tables"].shape[1] - 1)).clamp(min=0).long()
    at = row % bs
    last = n - queries + torch.arange(queries, device="cuda")
    sees = (row[:, None] <= last[..., None]) & own_place[:, None]
    if c["window"]:
        sees = sees & ((row[:, None] < c["first"]) | (row[:, None] > last[..., None] - c["window"]))
    k = st["k_cache"][block, :, at].float()
    x = st["q"].float().view(seqs, queries, kv, heads // kv, d).permute(0, 2, 1, 3, 4).reshape(seqs, kv, -1, d)
    score = (x @ k.permute(0, 2, 3, 1)).view(seqs, kv, queries, heads // kv, -1) * st["scale"]
    del k
    score = score.masked_fill(~sees[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = (score - top.masked_fill(top == -math.inf, 0)).exp()
    total = p.sum(-1, keepdim=True)
    p = (p / total.masked_fill(total == 0, 1)).view(seqs, kv, queries * (heads // kv), -1)
    v = st["v_cache"][block, :, at].float()
    o = (p @ v.permute(0, 2, 1, 3)).view(seqs, kv, queries, heads // kv, d).permute(0, 2, 1, 3, 4)
    return o.reshape(st["q"].shape).to(st["q"].dtype), p, row, block, at


def _plain_weights(st, c):
    out, p, row, block, at = _attend(st, c)
    n = st["lens"].long()[:, None]
    seq, col = (row < n).nonzero(as_tuple=True)
    block, at = block[seq, col], at[seq, col]
    w = p.sum(2).transpose(1, 2)[seq, col]  # [rows][kv_heads]
    old = st["row_weights"][block, :, at]
    new = (row[seq, col] >= n[seq, 0] - c["queries"])[:, None]
    st["row_weights"][block, :, at] = torch.where(new, w, old + w)
    return out, st["row_weights"]


def _plain_evict(st, c):
    bs, width = c["block"], st["max_len"]
    n, keep = st["lens"].long(), st["keep"].long()
    i = torch.arange(width, device="cuda")
    block = st["tables"].gather(1, (i // bs).expand(len(n), -1)).clamp(min=0).long()
    w = st["row_weights"][block, :, i % bs].transpose(1, 2).double()  # [seqs][kv_heads][rows]
    w = torch.where(w.isnan(), -math.inf, w).clamp(-1e300, 1e300)
    stays = (i < c["first"]) | (i >= n[:, None] - c["last"])
    w = torch.where(stays[:, None], math.inf, w)
    w = torch.where((i < n[:, None])[:, None], w, -math.inf)
    order = w.sort(dim=-1, descending=True, stable=True)[1]
    kept = torch.zeros_like(w, dtype=torch.bool).scatter_(-1, order, (i < keep[:, None])[:, None].expand_as(w))
    seq, head, src = kept.nonzero(as_tuple=True)
    dst = (kept.cumsum(-1) - 1)[seq, head, src]
    here = st["tables"][seq, src // bs].long(), head, src % bs
    there = st["tables_out"][seq, dst // bs].long(), head, dst % bs
    for name in ("k_cache", "v_cache", "row_weights", "k_params", "v_params"):
        if name in st:
            st[name][there] = st[name][here]
    st["lens_out"].copy_(st["keep"])
    return _evicted(st)


def _evicted(st):
    return tuple(st[name] for name in ("k_cache", "v_cache", "row_weights", "lens_out", "k_params", "v_params") if name in st)


def _plain_verify(st, c):
    b, q, v = c["seqs"], c["drafts"], c["vocab"]
    seq = torch.arange(b, device="cuda")
    nd = st["num_drafts"].long() if c["ragged"] else torch.full((b,), q, device="cuda")
    x = st["tokens"].long()
    p = st["target"][:, :q].gather(-1, x[..., None])[..., 0].double()
    qx = st["draft"].gather(-1, x[..., None])[..., 0].double() if st["draft"] is not None else torch.ones_like(p)
    good = (st["uniforms"][:, :q].double() * qx < p) & (torch.arange(q, device="cuda") < nd[:, None])
    a = good.long().cumprod(-1).sum(-1)
    r = st["target"][seq, a].double()
    taken = a < nd
    at = a.clamp(max=q - 1)
    if st["draft"] is not None:
        r = torch.where(taken[:, None], (r - st["draft"][seq, at].double()).clamp(min=0), r)
    else:
        r[seq, x[seq, at]] = torch.where(taken, 0.0, r[seq, x[seq, at]])
    r = torch.where(r.sum(-1, keepdim=True) > 0, r, st["target"][seq, a].double())
    upto = r.cumsum(-1)
    token = (upto <= st["uniforms"][:, q:].double() * upto[:, -1:]).sum(-1)
    i = torch.arange(q + 1, device="cuda")
    padded = torch.cat([x, x[:, :1]], 1)
    tokens = torch.where(i < a[:, None], padded, torch.where(i == a[:, None], token[:, None], -1))
    st["out_tokens"].copy_(tokens)
    st["accepted"].copy_(a)
    st["lens_out"].copy_(st["lens"].long() - (nd - a))
    return st["out_tokens"], st["accepted"], st["lens_out"]


# ------------------------------------------------------ the framework's calls


def run(st):
    c = st["case"]
    if c["kind"] == "evict" and c["place"] == "same":
        st["row_weights"].copy_(st["saved"])  # as accumulated: a pass in place leaves others behind
    if not own:
        if c["kind"] == "sinks":
            return _attend(st, c)[0]
        return {"weights": _plain_weights, "evict": _plain_evict, "verify": _plain_verify}[c["kind"]](st, c)
    import paged_kv_cache_29_gb300 as pa
    if c["kind"] == "verify":
        pa.pa_verify_draft(st["target"], st["draft"], st["tokens"], st["uniforms"], st["out_tokens"], st["accepted"],
                           num_drafts=st["num_drafts"], context_lens=st["lens"], lens_out=st["lens_out"])
        return st["out_tokens"], st["accepted"], st["lens_out"]
    if c["kind"] == "evict":
        if "workspace" not in st:  # scratch that a program keeps beside its pool
            need = pa.pa_evict_workspace_size(c["seqs"], c["kv_heads"], st["max_len"])
            st["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        pa.pa_evict(st["k_cache"], st["v_cache"], st["row_weights"], st["tables"], st["lens"], st["keep"], st["tables_out"], st["lens_out"],
                    st["max_len"], num_sinks=c["first"], num_recent=c["last"], k_params=st.get("k_params"), v_params=st.get("v_params"),
                    workspace=st["workspace"])
        return _evicted(st)
    sizes = (c["seqs"], c["queries"], c["heads"], c["head_dim"], st["max_len"])
    if c["kind"] == "sinks":
        if "workspace" not in st:
            st["workspace"] = torch.empty(max(pa.pa_decode_workspace_size_multi(*sizes), 16), dtype=torch.uint8, device="cuda")
        pa.pa_decode_sinks(st["q"], st["k_cache"], st["v_cache"], st["tables"], st["lens"], st["scale"], c["window"], c["first"], st["out"],
                           st["max_len"], workspace=st["workspace"])
        return st["out"]
    if "workspace" not in st:
        st["workspace"] = torch.empty(max(pa.pa_decode_workspace_size_weights(*sizes), 16), dtype=torch.uint8, device="cuda")
    pa.pa_decode_weights(st["q"], st["k_cache"], st["v_cache"], st["tables"], st["lens"], st["scale"], st["out"], st["row_weights"], st["max_len"],
                         workspace=st["workspace"])
    return st["out"], st["row_weights"]


# --------------------------------------------------------------- 64 bits


def _exact_rows(st, c, name, s, n):
    """Rows 0 .. n - 1 of sequence s of a pool, [kv_heads][n][...]."""
    blocks = st["tables"][s, : -(-n // c["block"])].long()
    return st[name][blocks].transpose(0, 1).flatten(1, 2)[:, :n]


def _exact_attention(st, c):
    seqs, queries, group = c["seqs"], c["queries"], c["heads"] // c["kv_heads"]
    out = torch.zeros(seqs, queries, c["heads"], c["head_dim"], dtype=torch.float64, device="cuda")
    q = st["q"].double().view(out.shape)
    total = st["row_weights"].double()
    for s, n in enumerate(_lens(c)):
        if n == 0:
            continue
        k, v = (_exact_rows(st, c, name, s, n).double() for name in ("k_cache", "v_cache"))
        new = torch.zeros(c["kv_heads"], n, dtype=torch.float64, device="cuda")
        for j in range(queries):
            end = n - queries + j + 1
            begin = max(0, end - c["window"]) if c["window"] else 0
            see = torch.cat([torch.arange(min(c["first"], begin)), torch.arange(begin, end)]).cuda()
            x = q[s, j].view(c["kv_heads"], group, -1)
            w = torch.softmax(torch.einsum("hgd,hnd->hgn", x, k[:, see]) * st["scale"], -1)
            out[s, j] = torch.einsum("hgn,hnd->hgd", w, v[:, see]).reshape(c["heads"], -1)
            new[:, see] += w.sum(1)
        if c["kind"] == "weights":
            i = torch.arange(n, device="cuda")
            block, at = st["tables"][s, i // c["block"]].long(), i % c["block"]
            total[block[: n - queries], :, at[: n - queries]] += new[:, : n - queries].t()
            total[block[n - queries:], :, at[n - queries:]] = new[:, n - queries:].t()
    out = out.view(st["out"].shape)
    return (out, total) if c["kind"] == "weights" else out


def _exact_evict(st, c):
    names = [n for n in ("k_cache", "v_cache", "row_weights", "k_params", "v_params") if n in st]
    out = {n: (st[n].clone() if not st[n].is_floating_point() else st[n].double()) for n in names}
    bs, lens = c["block"], _lens(c)
    for s, n in enumerate(lens):
        keep = _keep(c, n)
        begin, end = min(n, c["first"]), max(min(n, c["first"]), n - c["last"])
        more = keep - begin - (n - end)
        w = _exact_rows(st, c, "row_weights", s, n)
        j = torch.arange(keep, device="cuda")
        to_block, to_at = st["tables_out"][s, j // bs].long(), j % bs
        # Candidates above the border value all stay, those at it from the lowest index on.
        free = w[:, begin:end]
        stay = torch.ones_like(w, dtype=torch.bool)
        if more < end - begin:
            border = free.sort(-1, descending=True)[0][:, more - 1: more] if more else torch.full((w.shape[0], 1), math.inf, device="cuda")
            above, level = free > border, free == border
            stay[:, begin:end] = above | (level & (level.cumsum(-1) <= more - above.sum(-1, keepdim=True)))
        for name in names:
            rows = _exact_rows(st, c, name, s, n)
            moved = rows[stay].unflatten(0, (rows.shape[0], keep))  # [kv_heads][keep][...]
            out[name][to_block, :, to_at] = moved.transpose(0, 1).to(out[name].dtype)
    kept = torch.tensor([_keep(c, n) for n in lens], dtype=torch.int32, device="cuda")
    return (out["k_cache"], out["v_cache"], out["row_weights"], kept, *(out[n] for n in names[3:]))


def _exact_verify(st, c):
    tokens, accepted, lens = [], [], []
    for s in range(c["seqs"]):
        nd = int(st["num_drafts"][s]) if c["ragged"] else c["drafts"]
        u, x = st["uniforms"][s].double().tolist(), st["tokens"][s].tolist()
        a, rest = 0, st["target"][s, nd].double()
        while a < nd:
            p = st["target"][s, a].double()
            q = torch.zeros_like(p).index_fill_(0, st["tokens"][s, a: a + 1].long(), 1.0) if st["draft"] is None else st["draft"][s, a].double()
            if not u[a] * float(q[x[a]]) < float(p[x[a]]):
                rest = torch.where(p > q, p - q, 0.0)
                rest = rest if float(rest.sum()) > 0 else p
                break
            a += 1
        border = u[c["drafts"]] * float(rest.sum())
        token = int(torch.searchsorted(rest.cumsum(0), torch.tensor([border], dtype=torch.float64, device="cuda"), right=True))
        tokens.append(x[:a] + [token] + [-1] * (c["drafts"] - a))
        accepted.append(a)
        lens.append(int(st["lens"][s]) - (nd - a))
    return tuple(torch.tensor(v, dtype=torch.int32, device="cuda") for v in (tokens, accepted, lens))


def exact(c, seed):
    st = prepare(c, seed)
    if c["kind"] == "verify":
        return _exact_verify(st, c)
    if c["kind"] == "evict":
        return _exact_evict(st, c)
    return _exact_attention(st, c)
