"""The failure test of pa_decode_weights, without a GPU: what it refuses."""
import pytest

from paged_kv_cache_29_gb300 import _binding as pa
from test_cache_rows_cpu import INVALID, P, SIZES, WORKSPACE, lib  # noqa: F401 (a fixture)


@pytest.mark.parametrize("kw,tile,status", [(dict(), -1, INVALID), (dict(err=None), 3, INVALID), (dict(rw=None), 3, INVALID), (dict(), 3, WORKSPACE),
                                            (dict(B=0), 3, pa.PA_OK)])
def test_withheld_tile_of_weights_refuses(lib, kw, tile, status):  # noqa: F811
    a = dict(q=P, k=P, v=P, bt=P, cl=P, scale=0.1, out=P, rw=P, **SIZES)
    a.update(err=P)
    a.update(kw)
    assert lib.pa_test_withhold_tile_weights(*a.values(), tile, None) == status
