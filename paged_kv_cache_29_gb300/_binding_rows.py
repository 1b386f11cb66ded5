"""Binding of the calls that say which rows of a cache count: attention to a window and
the first rows, accumulated row weights, eviction by them, and verification of drafts.
Arguments, streams, workspaces and errors as in _binding."""
from . import _binding as _b


def pa_decode_workspace_size_weights(num_seqs: int, num_queries: int, num_heads: int,
                                     head_dim: int, max_context_len: int) -> int:
    return int(_b.lib().pa_decode_workspace_size_weights(num_seqs, num_queries, num_heads, head_dim,
                                                         max_context_len))


def pa_evict_workspace_size(num_seqs: int, num_kv_heads: int, max_context_len: int) -> int:
    return int(_b.lib().pa_evict_workspace_size(num_seqs, num_kv_heads, max_context_len))


def _rows_args(q, k_cache, v_cache, block_tables, context_lens, out, dev):
    """Pointers and sizes that pa_decode_sinks and pa_decode_weights share."""
    import torch
    kc = _b._arg("k_cache", k_cache, dev, None, 4)
    dt = k_cache.dtype
    vc = _b._arg("v_cache", v_cache, dev, dt)
    qp = _b._arg("q", q, dev, dt)
    op = _b._arg("out", out, dev, dt)
    bt = _b._arg("block_tables", block_tables, dev, torch.int32, 2)
    cl = _b._arg("context_lens", context_lens, dev, torch.int32, 1)
    pool = k_cache.shape
    nb, hkv, bs, d = pool
    shape = q.shape
    if len(shape) == 3:
        (B, hq, dq), Q = shape, 1
    elif len(shape) == 4:
        B, Q, hq, dq = shape
    else:
        raise ValueError(f"q must have 3 or 4 dimensions, got {len(shape)}")
    rows, mb = block_tables.shape
    if dq != d or out.shape != shape or v_cache.shape != pool or rows != B or context_lens.numel() != B:
        raise ValueError("shape mismatch between q/out/block_tables/context_lens and the caches")
    return (qp, kc, vc, bt, cl), op, (B, Q, hq, hkv, d, bs, nb, mb), _b._plain_dtype_code(k_cache)


def pa_decode_sinks(q, k_cache, v_cache, block_tables, context_lens, scale, window, num_sinks, out,
                    max_context_len, workspace=None, error_word=None, stream=None) -> None:
    """Decode attention to the last `window` rows and to the first `num_sinks`
    rows, which stay visible. q/out: [B][Hq][D], or [B][Q][Hq][D] for the last Q
    tokens of every sequence (token j sits at row r = n - Q + j and attends to the
    rows i <= r with i < num_sinks or i > r - window); fp32 or bf16 like the caches.
    workspace: a CUDA tensor of at least
    pa_decode_workspace_size_multi(B, Q, Hq, D, max_context_len) bytes; when None,
    one is taken from torch's caching allocator for this call, on its stream."""
    import torch
    dev = torch.cuda.current_device()
    ptrs, op, sizes, code = _rows_args(q, k_cache, v_cache, block_tables, context_lens, out, dev)
    bound, window = _b._int32("max_context_len", max_context_len), _b._int32("window", window)
    num_sinks = _b._int32("num_sinks", num_sinks)
    if workspace is None:
        need = _b.pa_decode_workspace_size_multi(sizes[0], sizes[1], sizes[2], sizes[4], bound)
        workspace = _b._scratch(need, stream, q.device)
    ws = _b._arg("workspace", workspace, dev)
    rc = _b.lib().pa_decode_sinks(*ptrs, float(scale), window, num_sinks, op, *sizes, bound, code, ws,
                                  workspace.numel() * workspace.element_size(),
                                  _b._opt_arg("error_word", error_word, dev, torch.int32),
                                  _b._stream_on(stream, dev))
    if rc != _b.PA_OK:
        raise _b.PagedAttentionError(rc, "pa_decode_sinks")


def pa_decode_weights(q, k_cache, v_cache, block_tables, context_lens, scale, out, row_weights,
                      max_context_len, workspace=None, error_word=None, stream=None) -> None:
    """Decode attention (q/out as in pa_decode_sinks, every row up to the token's own)
    that adds each row's attention weight, summed over the query heads of its KV
    head and the Q tokens, to row_weights (fp32 [NB][Hkv][bs]); the rows of the last
    Q tokens, whose slots no other sequence of the batch holds, begin their sums. What tokens that
    are rejected afterwards added to earlier rows stays. workspace: at least
    pa_decode_workspace_size_weights(B, Q, Hq, D, max_context_len) bytes; None as in
    pa_decode_sinks."""
    import torch
    dev = torch.cuda.current_device()
    ptrs, op, sizes, code = _rows_args(q, k_cache, v_cache, block_tables, context_lens, out, dev)
    rw = _b._arg("row_weights", row_weights, dev, torch.float32, 3)
    if row_weights.shape != k_cache.shape[:3]:
        raise ValueError("row_weights must be [NB][Hkv][bs]")
    bound = _b._int32("max_context_len", max_context_len)
    if workspace is None:
        need = pa_decode_workspace_size_weights(sizes[0], sizes[1], sizes[2], sizes[4], bound)
        workspace = _b._scratch(need, stream, q.device)
    ws = _b._arg("workspace", workspace, dev)
    rc = _b.lib().pa_decode_weights(*ptrs, float(scale), op, rw, *sizes, bound, code, ws,
                                    workspace.numel() * workspace.element_size(),
                                    _b._opt_arg("error_word", error_word, dev, torch.int32),
                                    _b._stream_on(stream, dev))
    if rc != _b.PA_OK:
        raise _b.PagedAttentionError(rc, "pa_decode_weights")


def pa_evict(k_cache, v_cache, row_weights, block_tables, context_lens, keep_lens, out_tables,
             lens_out, max_context_len, num_sinks=0, num_recent=0, k_params=None, v_params=None,
             workspace=None, error_word=None, stream=None) -> None:
    """Cuts each sequence to keep_lens[s] rows (int32 [B]): under each KV head the
    first num_sinks and the last num_recent rows stay, and of the others those with
    the largest row_weights (fp32 [NB][Hkv][bs]; of equal ones the first). They move,
    in their order, to the first rows of out_tables (block_tables itself: in place),
    with their weights and params. lens_out (int32 [B], may be context_lens) gets
    the new lengths.

    Pools as the decode calls take them; INT8 caches with k_params/v_params their fp32
    scales ([NB][Hkv][bs]), INT4 ones (uint8 codes [NB][Hkv][bs][D / 2]) with bf16
    pairs ([NB][Hkv][bs][2]). Blocks shared with other sequences: out_tables with
    blocks of the sequence's own. workspace: at least
    pa_evict_workspace_size(B, Hkv, max_context_len) bytes; None as in pa_decode_sinks."""
    import torch
    dev = torch.cuda.current_device()
    kc = _b._arg("k_cache", k_cache, dev, None, 4)
    vc = _b._arg("v_cache", v_cache, dev, k_cache.dtype)
    code = _b._plain_dtype_code(k_cache)
    nb, hkv, bs, d = pool = k_cache.shape
    if k_cache.dtype is torch.uint8 and k_params is not None:
        code, d = 4, 2 * d
    kp = vp = None
    if code >= 3:
        want = (torch.bfloat16, (nb, hkv, bs, 2)) if code == 4 else (torch.float32, (nb, hkv, bs))
        kp, vp = _b._arg("k_params", k_params, dev, want[0]), _b._arg("v_params", v_params, dev, want[0])
        if k_params.shape != want[1] or v_params.shape != want[1]:
            raise ValueError("k_params and v_params must hold 4 bytes per row: [NB][Hkv][bs] scales or [NB][Hkv][bs][2] pairs")
    elif k_params is not None or v_params is not None:
        raise ValueError("k_params and v_params belong to INT8 and INT4 caches")
    rw = _b._arg("row_weights", row_weights, dev, torch.float32, 3)
    bt = _b._arg("block_tables", block_tables, dev, torch.int32, 2)
    ot = _b._arg("out_tables", out_tables, dev, torch.int32, 2)
    cl = _b._arg("context_lens", context_lens, dev, torch.int32, 1)
    kl = _b._arg("keep_lens", keep_lens, dev, torch.int32, 1)
    lo = _b._arg("lens_out", lens_out, dev, torch.int32, 1)
    B, mb = block_tables.shape
    if v_cache.shape != pool or row_weights.shape != pool[:3] or out_tables.shape != block_tables.shape \
            or context_lens.numel() != B or keep_lens.numel() != B or lens_out.numel() != B:
        raise ValueError("shape mismatch between the caches, row_weights, the tables and the lengths")
    bound = _b._int32("max_context_len", max_context_len)
    if workspace is None:
        workspace = _b._scratch(pa_evict_workspace_size(B, hkv, bound), stream, k_cache.device)
    ws = _b._arg("workspace", workspace, dev)
    rc = _b.lib().pa_evict(kc, vc, kp, vp, rw, bt, cl, kl, ot, lo, _b._int32("num_sinks", num_sinks),
                           _b._int32("num_recent", num_recent), B, hkv, d, bs, nb, mb, bound, code, ws,
                           workspace.numel() * workspace.element_size(),
                           _b._opt_arg("error_word", error_word, dev, torch.int32),
                           _b._stream_on(stream, dev))
    if rc != _b.PA_OK:
        raise _b.PagedAttentionError(rc, "pa_evict")


def _probs_arg(name, t, dev):
    """Pointer and (sequence, row) strides of fp32 probabilities [B][rows][V] whose
    rows are contiguous and may lie any distance apart."""
    import torch
    try:
        if t.get_device() == dev and t.dtype is torch.float32:
            seq, row, one = t.stride()
            if one == 1:
                return t.data_ptr(), seq, row
    except (AttributeError, ValueError):
        pass
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be {torch.float32}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must have 3 dimensions, got {t.dim()}")
    _b._check_device(None, t)
    seq, row, one = t.stride()
    if one != 1 and t.shape[2] > 1:
        raise ValueError(f"{name}: the values of a row must be contiguous")
    return t.data_ptr(), seq, row


def pa_verify_draft(target_probs, draft_probs, draft_tokens, uniforms, out_tokens, num_accepted,
                    num_drafts=None, context_lens=None, lens_out=None, error_word=None,
                    stream=None) -> None:
    """Accepts or rejects drafted tokens against the target's probabilities, and draws
    one more token, from given random numbers. target_probs: fp32 [B][Q + 1][V];
    draft_probs: fp32 [B][Q][V], or None where the drafts were looked up, not
    drawn; draft_tokens: int32 [B][Q]; uniforms: fp32 [B][Q + 1] in [0, 1), the last of
    a row for the drawn token. num_drafts: int32 [B] (None: Q each).
    out_tokens: int32 [B][Q + 1], the accepted tokens, the drawn one, then -1;
    num_accepted: int32 [B]. With context_lens, the rows cached with all the drafts,
    lens_out (may be context_lens) gets the lengths without the rejected ones."""
    import torch
    dev = torch.cuda.current_device()
    tp, t_seq, t_row = _probs_arg("target_probs", target_probs, dev)
    B, rows, V = target_probs.shape
    Q = rows - 1
    dp, d_seq, d_row = (None, 0, 0) if draft_probs is None else _probs_arg("draft_probs", draft_probs, dev)
    dt = _b._arg("draft_tokens", draft_tokens, dev, torch.int32, 2)
    un = _b._arg("uniforms", uniforms, dev, torch.float32, 2)
    ot = _b._arg("out_tokens", out_tokens, dev, torch.int32, 2)
    na = _b._arg("num_accepted", num_accepted, dev, torch.int32, 1)
    nd = _b._opt_arg("num_drafts", num_drafts, dev, torch.int32, 1)
    cl = _b._opt_arg("context_lens", context_lens, dev, torch.int32, 1)
    lo = _b._opt_arg("lens_out", lens_out, dev, torch.int32, 1)
    if Q < 0 or draft_tokens.shape != (B, Q) or uniforms.shape != (B, rows) or out_tokens.shape != (B, rows) \
            or (draft_probs is not None and draft_probs.shape != (B, Q, V)) or num_accepted.numel() != B \
            or any(t is not None and t.numel() != B for t in (num_drafts, context_lens, lens_out)):
        raise ValueError("shape mismatch between the probabilities, the drafted tokens and the outputs")
    rc = _b.lib().pa_verify_draft(tp, t_seq, t_row, dp, d_seq, d_row, dt, nd, un, ot, na, cl, lo, B, Q,
                                  V, _b._opt_arg("error_word", error_word, dev, torch.int32),
                                  _b._stream_on(stream, dev))
    if rc != _b.PA_OK:
        raise _b.PagedAttentionError(rc, "pa_verify_draft")
