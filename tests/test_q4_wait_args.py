"""zf_q4_decode_attn_wait_test without a GPU: it refuses what zf_q4_decode_attn refuses, and limits out of range, before
anything is launched."""
import ctypes

import pytest

from tests import helpers as H
from tests.test_step_args import BAD_CACHES, _desc


def test_wait_test_refuses():
    zf = H.zf_module()
    f = zf.lib().zf_q4_decode_attn_wait_test

    def call(desc, batch=2, tokens=1, hq=8, q=0x10000, ws=0x40000, scale=0.1, limit=1_000_000):
        return f(ctypes.byref(desc), q, batch, tokens, hq, 0x50000, 4, 0x60000, scale, 0x20000, 0x30000, ws, 1 << 30, limit, None)
    for kw, code in BAD_CACHES:
        assert call(_desc(zf, **kw)) == code, kw
    d = _desc(zf)
    for kw in (dict(limit=0), dict(limit=999), dict(limit=2_000_000_001), dict(limit=2 ** 64 - 1), dict(batch=-1), dict(batch=4097),
               dict(tokens=0), dict(tokens=65), dict(hq=7), dict(q=None), dict(q=0x10004), dict(ws=None), dict(scale=float("nan"))):
        assert call(d, **kw) == -1, kw
    assert call(d, batch=0) == 0
    assert call(d, batch=0, limit=999) == -1


def test_binding_checks_the_query():
    import torch
    zf = H.zf_module()
    c = zf.Q4Cache(4, 2, 16, device="cpu")
    table, lens = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="a CUDA device"):
        zf.q4_decode_attn_wait_test(c, torch.zeros(3, 1, 8, 128, dtype=torch.int16), table, lens)
    with pytest.raises(ValueError, match="q: dtype"):
        zf.q4_decode_attn_wait_test(c, torch.zeros(3, 1, 8, 128), table, lens)
