"""pa_decode_weights where a wait of the tile ring gives up: nothing that the workspace
held before reaches the row weights."""
import numpy as np
import pytest
import torch

import cache_rows_reference as ref
import paged_kv_cache_29_gb300 as pkg
from paged_kv_cache_29_gb300 import _binding as pa
from test_gpu_decode_rows import Run, start_weights

pytestmark = pytest.mark.gpu


def withhold(run, w, workspace, tile):
    """pa_decode_weights whose CTA 0 withholds a tile: the waiting consumer gives up after about 2 s."""
    ptr = lambda t: t.data_ptr()
    nb, hkv, bs, d = run.dk.shape
    out = run.out()
    rc = pa.lib().pa_test_withhold_tile_weights(
        ptr(run.dq), ptr(run.dk), ptr(run.dv), ptr(run.table), ptr(run.n), run.scale, ptr(out), ptr(w), len(run.lens), run.Q, run.group * hkv, hkv,
        d, bs, nb, run.table.shape[1], run.bound, 0 if run.dtype == "f32" else 1, ptr(workspace), workspace.numel() * 4, ptr(run.err), tile,
        torch.cuda.current_stream().cuda_stream)
    assert rc == pa.PA_OK


@pytest.mark.parametrize("shape,lens", [
    (("bf16", 4, 1, 128, 16), [1300, 530, 40] * 40),   # several items a CTA, sequences over several CTAs
    (("bf16", 4, 5, 128, 16), [1300, 700, 90] * 10),   # three column groups
    (("f32", 4, 1, 64, 16), [1300, 530, 40] * 40),
    (("bf16", 4, 1, 128, 16), [500, 300, 90] * 2),     # one partition each: added at the items' ends
], ids=str)
def test_weights_of_a_call_that_gave_up_are_this_calls_or_as_before(shape, lens):
    run = Run(shape, lens, hkv=4, seed=31)
    start = start_weights(run.cache)
    _, clean = run.weights(start)
    assert int(run.err.item()) == 0
    need = pkg.pa_decode_workspace_size_weights(len(lens), run.Q, run.group * run.hkv, run.D, run.bound)
    ws = torch.ones((need + 3) // 4, device="cuda")    # states and scores of an earlier call, all usable
    w = torch.from_numpy(start).cuda()
    withhold(run, w, ws, 5)
    torch.cuda.synchronize()
    assert int(run.err.item()) == pa.PA_DEVERR_TIMEOUT
    got, left = w.cpu().numpy(), 0
    for s, n in enumerate(lens):
        g, c, b = (ref.slot_rows(x, run.cache.table[s], n, run.bs) for x in (got, clean, start))
        for h in range(run.hkv):
            as_before = np.array_equal(g[:, h], b[:, h])
            assert as_before or np.array_equal(g[:, h], c[:, h]), (s, h)
            left += as_before
    assert left > 0
    # The same tensors and workspace again: exact, nothing flagged.
    run.err.zero_()
    out, again = run.weights(start, workspace=ws)
    run.check(out)
    assert np.array_equal(again, clean) and int(run.err.item()) == 0
