"""Numbers past 32 bits are refused by the 4-bit calls of the binding; cut to 32 bits, a
window of 2^32 + 5 rows would be one of 5."""
import pytest
import torch

from paged_kv_cache_29_gb300 import _binding as pa
from test_int4_cpu import _dev, _pool, _Shapes, no_library  # noqa: F401


@pytest.mark.parametrize("kw,name", [(dict(window=2 ** 32 + 5), "window"), (dict(window=2 ** 31), "window"),
                                     (dict(window=-2 ** 32), "window"), (dict(bound=2 ** 32 + 64), "max_context_len")])
@pytest.mark.parametrize("own_workspace", [False, True])
def test_decode(no_library, kw, name, own_workspace):  # noqa: F811
    z = _Shapes()
    q = _dev((z.B, z.hq, z.d))
    ws = _dev((4096,), torch.uint8) if own_workspace else None
    kw = dict(kw)
    with pytest.raises(ValueError, match=name):
        pa.pa_decode_int4(q, *_pool(z), _dev((z.B, 4), torch.int32), _dev((z.B,), torch.int32), 0.1, q, kw.pop("bound", 64),
                          workspace=ws, **kw)


def test_gather(no_library):  # noqa: F811
    z = _Shapes()
    rows = _dev((z.B, z.hkv, z.d))
    with pytest.raises(ValueError, match="max_context_len"):
        pa.pa_gather_int4(*_pool(z), _dev((z.B, 4), torch.int32), _dev((z.B,), torch.int32), _dev((z.B,), torch.int64), rows, rows,
                          2 ** 32 + 64)
