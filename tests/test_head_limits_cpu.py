"""More heads than the 4-bit and the norm and rotation calls' 32-bit arithmetic
holds are refused on the host, with nothing enqueued."""
import ctypes

import pytest

from paged_kv_cache_29_gb300 import _binding as pa
from test_int4_cpu import NORM, UNSUPPORTED, WORKSPACE, _append, _decode, _gather, _norm, lib  # noqa: F401

MOST = 1 << 20


@pytest.mark.parametrize("heads", [MOST + 1, 1 << 28, 2 ** 31 - 1])
def test_too_many_heads(lib, heads):  # noqa: F811
    wide = 1 << 50
    assert _append(lib, hkv=heads) == UNSUPPORTED
    assert _gather(lib, hkv=heads) == UNSUPPORTED
    assert _decode(lib, hq=heads, hkv=heads, nb=1) == UNSUPPORTED
    assert _norm(lib, num_heads=heads, q_stride=wide, q_out_stride=wide) == UNSUPPORTED
    assert _norm(lib, num_kv_heads=heads, k_stride=wide, k_out_stride=wide) == UNSUPPORTED
    args = pa._NormRopeArgs(**{**NORM, "num_kv_heads": heads, "k_stride": wide})
    assert lib.pa_norm_rope_append(ctypes.byref(args), 1 << 20, wide, 1 << 20, 1 << 20, 1 << 20, 16, 4, None, None) == UNSUPPORTED
    assert lib.pa_norm_rope_append_int4(ctypes.byref(args), 1 << 20, wide, *[1 << 20] * 5, 16, 4, None, None) == UNSUPPORTED


def test_the_most_heads_are_taken(lib):  # noqa: F811
    """No token, or no workspace, ends the call behind the check."""
    assert _append(lib, hkv=MOST, T=0) == pa.PA_OK
    assert _gather(lib, hkv=MOST, B=0) == pa.PA_OK
    assert _norm(lib, num_heads=MOST, num_kv_heads=MOST, num_tokens=0) == pa.PA_OK
    assert _decode(lib, hq=MOST, hkv=MOST, nb=1) == WORKSPACE
