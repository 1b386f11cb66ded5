"""pa_verify_draft and probabilities that are not finite: an infinite r is flagged, a NaN or
negative one counts as 0."""
import numpy as np
import pytest
import torch

import paged_kv_cache_29_gb300 as pkg
from paged_kv_cache_29_gb300 import _binding as pa

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("V", [5, 600, 50021])
@pytest.mark.parametrize("p,q,flagged", [(INF, 0.0, True), (0.1, -INF, True), (INF, 0.3, True), (INF, INF, False), (-INF, 0.0, False), (0.1, INF, False),
                                         (NAN, 0.0, False), (0.1, NAN, False), (INF, NAN, False), (-INF, -INF, False)])
def test_one_value_that_is_not_finite(V, p, q, flagged):
    """A rejected draft; beside it a sequence of finite values and one that accepts all."""
    at, x, other = V - 1, 1, 2
    target = np.zeros((3, 2, V), np.float32)
    target[:, :, other], target[:, 1, 3] = 0.5, 0.5
    target[2, 0, x] = 1.0                              # accepted: its last row holds the value
    draft = np.zeros((3, 1, V), np.float32)
    draft[:, 0, x] = 1.0
    target[0, 0, at], draft[0, 0, at] = p, q
    target[2, 1, at] = p
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, acc = torch.full((3, 2), -9, dtype=torch.int32, device="cuda"), torch.full((3,), -9, dtype=torch.int32, device="cuda")
    dev = lambda a: torch.from_numpy(a).cuda()
    pkg.pa_verify_draft(dev(target), dev(draft), torch.full((3, 1), x, dtype=torch.int32, device="cuda"),
                        torch.tensor([[0.5, 0.25]] * 3, device="cuda"), out, acc, error_word=err)
    last = p == INF                                    # of the sequence that accepts, without q
    assert out[1].tolist() == [other, -1] and acc[1] == 0
    assert (out[0].tolist(), int(acc[0])) == (([-9, -9], -9) if flagged else ([other, -1], 0))
    assert (out[2].tolist(), int(acc[2])) == (([-9, -9], -9) if last else ([x, other], 1))
    assert int(err.item()) == (pa.PA_DEVERR_TOKEN if flagged or last else 0)
