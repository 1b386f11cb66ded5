"""Decode calls without a workspace on a stream that is not torch's current one,
while the current one fills every tensor that the allocator gives it."""
import pytest
import torch

from gpu_helpers import DeviceStep
from paged_kv_cache_29_gb300 import _binding as pa
from paged_kv_cache_29_gb300 import workloads as wl
from test_gpu_int4 import Batch, host, value

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["torch stream", "raw handle"])
def side(request):
    stream = torch.cuda.Stream()
    yield stream, (stream if request.param == "torch stream" else stream.cuda_stream)
    torch.cuda.synchronize()


def _fill(nbytes):
    for _ in range(4):
        torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")


def test_int4_scratch_is_not_handed_out_under_a_running_call(side):
    stream, handle = side
    b = Batch([5000, 40, 3000, 2200] * 16, hq=8, hkv=2, seed=50).upload()
    need = pa.pa_decode_workspace_size_multi(len(b.lens), 1, 8, 128, b.mcl)
    want = torch.empty_like(b.out)
    pa.pa_decode_int4(b.dq, *b.dpools, b.dtable, b.dlens, b.scale, want, b.mcl)
    _fill(need)
    stream.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        pa.pa_decode_int4(b.dq, *b.dpools, b.dtable, b.dlens, b.scale, b.out, b.mcl, error_word=b.err, stream=handle)
        _fill(need)
    torch.cuda.synchronize()
    assert int(b.err.item()) == 0
    assert torch.equal(b.out, want)
    b.check(value(host(want))[:, None], skip=set(range(4, 64)))


def test_decode_scratch_is_not_handed_out_under_a_running_call(side):
    stream, handle = side
    step = wl.build_step("scratch", [1400, 30, 2100, 700] * 4, 8, 2, 128, seed=51)
    d = DeviceStep(step)
    d.append()
    need = d.workspace.numel()
    d.decode()
    want = d.out.clone()
    _fill(need)
    stream.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        pa.pa_decode(d.q, d.k_cache, d.v_cache, d.tables, d.lens, step.scale, d.out, step.max_context_len, error_word=d.err,
                     stream=handle)
        _fill(need)
    torch.cuda.synchronize()
    assert int(d.err.item()) == 0
    assert torch.equal(d.out, want)
