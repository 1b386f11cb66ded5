"""Lengths that one call writes on the device are those that the next call on the stream
reads, with nothing between the two: verification, eviction and every decode call that
plans its work from the lengths."""
import numpy as np
import pytest
import torch

import paged_kv_cache_29_gb300 as pkg
from paged_kv_cache_29_gb300 import _binding as pa
from test_gpu_decode_rows import Run, start_weights

pytestmark = pytest.mark.gpu

B, Q, V = 96, 3, 500


class Steps:
    def __init__(self, seed):
        r = np.random.default_rng(seed)
        self.run = run = Run(("bf16", 4, 1, 128, 16), [int(n) for n in r.integers(40, 900, B)], hkv=2, seed=seed)
        self.first = torch.tensor(run.lens, dtype=torch.int32).cuda()
        self.lens = self.first.clone()
        self.k, self.v, self.w = run.dk.clone(), run.dv.clone(), torch.from_numpy(start_weights(run.cache)).cuda()
        self.keep_of = [x.clone() for x in (self.k, self.v, self.w)]
        self.target = torch.full((B, Q + 1, V), 1.0 / V, device="cuda")
        self.tokens = torch.from_numpy(r.integers(0, V, (B, Q)).astype(np.int32)).cuda()
        self.uniforms = torch.from_numpy((r.random((B, Q + 1)) * 4 / V).astype(np.float32)).cuda()   # a quarter accepted
        self.new, self.accepted = torch.zeros(B, Q + 1, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
        self.budget = torch.from_numpy(r.integers(30, 600, B).astype(np.int32)).cuda()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.q = run.dq[:, 0]
        self.out = [torch.full_like(self.q, 7.0) for _ in range(6)]
        need = max(pkg.pa_decode_workspace_size_weights(B, 1, 8, 128, run.bound), pa.pa_decode_workspace_size_multi(B, 1, 8, 128, run.bound),
                   pkg.pa_evict_workspace_size(B, 2, run.bound))
        self.ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()

    def calls(self):
        r, o = self.run, self.out
        kw = dict(workspace=self.ws, error_word=self.err)
        args = (self.q, self.k, self.v, r.table, self.lens, r.scale)
        check = lambda: pkg.pa_verify_draft(self.target, None, self.tokens, self.uniforms, self.new, self.accepted, context_lens=self.lens,
                                            lens_out=self.lens, error_word=self.err)
        evict = lambda: pkg.pa_evict(self.k, self.v, self.w, r.table, self.lens, self.budget, r.table, self.lens, r.bound, 2, 8, **kw)
        return [check, lambda: pkg.pa_decode_weights(*args, o[0], self.w, r.bound, **kw),
                check, lambda: pkg.pa_decode_sinks(*args, 100, 4, o[1], r.bound, **kw),
                check, lambda: pa.pa_decode(*args, o[2], r.bound, **kw),
                evict, lambda: pkg.pa_decode_weights(*args, o[3], self.w, r.bound, **kw),
                check, evict, lambda: pa.pa_decode(*args, o[4], r.bound, **kw),
                check, check, lambda: pkg.pa_decode_sinks(*args, 30, 0, o[5], r.bound, **kw)]

    def state(self):
        torch.cuda.synchronize()
        assert int(self.err.item()) == 0
        return [x.clone() for x in (*self.out, self.w, self.lens, self.accepted, self.k.view(torch.int16), self.v.view(torch.int16))]

    def reset(self):
        for x, y in zip((self.k, self.v, self.w, self.lens), (*self.keep_of, self.first)):
            x.copy_(y)


@pytest.mark.parametrize("seed", [1, 2])
def test_calls_read_the_lengths_that_the_call_before_wrote(seed):
    st = Steps(seed)
    for call in st.calls():                            # one at a time
        call()
        torch.cuda.synchronize()
    want = st.state()
    # (Where all drafts are accepted and the budget is above the length, it stays.)
    assert (st.lens < st.first).sum() > B // 2 and len(set(st.accepted.tolist())) > 1
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call in st.calls():
            call()
    for turn in range(20):
        st.reset()
        if turn % 2:
            graph.replay()
        else:
            for call in st.calls():
                call()
        for a, b in zip(st.state(), want):
            assert torch.equal(a, b)
