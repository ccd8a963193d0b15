"""Chunk attention, sampling and the page calls without a GPU: what they refuse before anything is launched, in the
C ABI and in the binding, and pins of their oracle."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import zf_serve_oracle as R
from tests import helpers as H
from tests.test_step_args import BAD_CACHES, _desc


@pytest.fixture(scope="module")
def zf():
    return H.zf_module()


def _caller(f, names, good):
    def call(**kw):
        args = list(good)
        for k, v in kw.items():
            args[names.index(k)] = v
        return f(*args)
    return call


def test_chunk_attention_refuses(zf):
    f = zf.lib().zf_q4_chunk_attn
    d = _desc(zf)
    names = ["cache", "q", "rows", "batch", "hq", "start", "table", "max_pages", "lens", "scale", "window", "cap", "slopes",
             "out", "lse", "ws", "ws_bytes", "stream"]
    call = _caller(f, names, [ctypes.byref(d), 0x10000, 5, 2, 8, 0x20000, 0x30000, 4, 0x40000, 0.1, 0, 0.0, None, 0x50000,
                              0x60000, 0x70000, 1 << 30, None])
    for kw, code in BAD_CACHES:
        assert call(cache=ctypes.byref(_desc(zf, **kw))) == code, kw
    for kw in (dict(cache=None), dict(rows=-1), dict(batch=-1), dict(batch=4097), dict(hq=7), dict(hq=1), dict(hq=0),
               dict(max_pages=0), dict(max_pages=1 << 27), dict(window=-1), dict(cap=-1.0), dict(cap=1e-4), dict(cap=1e7),
               dict(cap=float("nan")), dict(cap=float("inf")), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(scale=1e38), dict(q=0x10008), dict(out=0x50004), dict(ws=0x70008), dict(start=0x20002),
               dict(table=0x30001), dict(lens=0x40003), dict(slopes=0x90002), dict(lse=0x60002),
               dict(rows=1 << 30, hq=16)):                             # more rows per kv head than are counted
        assert call(**kw) == -1, kw
    for name in ("q", "start", "table", "lens", "out", "lse", "ws"):
        assert call(**{name: None}) == -1, name
    assert call(cache=ctypes.byref(_desc(zf, k_scale=1e30)), scale=1e10) == -1
    assert call(rows=0) == 0 and call(batch=0) == 0
    size = zf.lib().zf_q4_chunk_attn_workspace_size
    for args in ((4097, 1, 8, 2, 16, 4), (1, -1, 8, 2, 16, 4), (1, 1, 7, 2, 16, 4), (1, 1, 8, 2, 24, 4), (1, 1, 8, 2, 256, 4),
                 (1, 1, 8, 2, 16, 0)):
        assert size(*args) == 0, args


def test_chunk_wait_test_refuses(zf):
    d = _desc(zf)
    names = ["cache", "q", "rows", "batch", "hq", "start", "table", "max_pages", "lens", "scale", "window", "cap", "slopes",
             "out", "lse", "ws", "ws_bytes", "limit", "stream"]
    call = _caller(zf.lib().zf_q4_chunk_attn_wait_test, names, [ctypes.byref(d), 0x10000, 5, 2, 8, 0x20000, 0x30000, 4, 0x40000,
                                                               0.1, 0, 0.0, None, 0x50000, 0x60000, 0x70000, 1 << 30, 1000000, None])
    for kw, code in BAD_CACHES:
        assert call(cache=ctypes.byref(_desc(zf, **kw))) == code, kw
    for kw in (dict(limit=0), dict(limit=999), dict(limit=2_000_000_001), dict(limit=2 ** 64 - 1), dict(batch=-1), dict(hq=7),
               dict(q=None), dict(ws=None), dict(scale=float("nan")), dict(window=-1), dict(batch=0, limit=999)):
        assert call(**kw) == -1, kw
    assert call(batch=0) == 0 and call(rows=0) == 0


def test_sampling_refuses(zf):
    names = ["rows", "vocab", "logits", "type", "stride", "uniform", "temp", "k", "p", "min_p", "tokens", "probs", "status",
             "stream"]
    call = _caller(zf.lib().zf_sample_tokens, names,
                   [2, 100, 0x1000, 0, 100, 0x2000, 0x2100, 0x2200, 0x2300, 0x2400, 0x2500, 0x3000, None, None])
    for kw in (dict(rows=-1), dict(rows=(1 << 20) + 1), dict(vocab=0), dict(vocab=(1 << 21) + 1, stride=1 << 22), dict(stride=99),
               dict(type=3), dict(type=-1), dict(logits=None), dict(logits=0x1002), dict(logits=0x1001, type=1),
               dict(uniform=None), dict(tokens=None), dict(uniform=None, tokens=None, probs=None)):
        assert call(**kw) == -1, kw
    for name in ("uniform", "temp", "k", "p", "min_p", "tokens", "probs", "status"):
        assert call(**{name: 0x4002}) == -1, name
    assert call(rows=0) == 0


def test_fork_refuses(zf):
    names = ["batch", "page", "max_pages", "lens", "held", "src", "dst", "n", "table", "free", "num_free", "pos", "out_lens",
             "out_held", "out_pos", "copy_src", "copy_dst", "status", "stream"]
    good = [2, 16, 4, 0x1000, 0x1100, 0x1200, 0x1300, 1, 0x2000, 0x3000, 8, 0x1400, 0x1500, 0x1600, 0x1700, 0x1800, 0x1900,
            None, None]
    call = _caller(zf.lib().zf_fork_requests, names, good)
    for kw in (dict(batch=-1), dict(batch=4097), dict(page=0), dict(page=24), dict(max_pages=0), dict(max_pages=1 << 27),
               dict(n=-1), dict(n=4097), dict(num_free=-1), dict(status=0x7001)):
        assert call(**kw) == -1, kw
    for name in ("lens", "held", "src", "dst", "table", "free", "pos", "out_lens", "out_held", "out_pos", "copy_src", "copy_dst"):
        assert call(**{name: None}) == -1 and call(**{name: 0x9002}) == -1, name
    assert call(page=256) == -2


def test_release_and_compact_refuse(zf):
    names = ["batch", "max_pages", "pool", "table", "lens", "held", "release", "free", "num_free", "pos", "out_lens", "out_held",
             "out_pos", "status", "ws", "ws_bytes", "stream"]
    call = _caller(zf.lib().zf_release_requests, names,
                   [2, 4, 100, 0x1000, 0x1100, 0x1200, 0x1300, 0x1400, 100, 0x1500, 0x1600, 0x1700, 0x1800, None, 0x2000, 1 << 20, None])
    for kw in (dict(batch=-1), dict(batch=4097), dict(max_pages=0), dict(pool=-1), dict(num_free=-1), dict(ws=None),
               dict(ws=0x2008), dict(status=0x7002)):
        assert call(**kw) == -1, kw
    for name in ("table", "lens", "held", "release", "free", "pos", "out_lens", "out_held", "out_pos"):
        assert call(**{name: None}) == -1 and call(**{name: 0x9002}) == -1, name
    assert call(batch=4096, max_pages=(1 << 18) + 1) == -2
    need = zf.lib().zf_release_requests_workspace_size(100)
    assert need >= 400 and call(ws_bytes=need - 1) == -3
    names = ["batch", "max_pages", "pool", "table", "held", "out", "free", "pos", "copy_src", "copy_dst", "status", "ws",
             "ws_bytes", "stream"]
    call = _caller(zf.lib().zf_compact_pages, names,
                   [2, 4, 100, 0x1000, 0x1100, 0x1200, 0x1300, 0x1400, 0x1500, 0x1600, None, 0x2000, 1 << 20, None])
    for kw in (dict(batch=-1), dict(batch=4097), dict(max_pages=0), dict(pool=-1), dict(ws=None), dict(ws=0x2008),
               dict(status=0x7002)):
        assert call(**kw) == -1, kw
    for name in ("table", "held", "out", "free", "pos", "copy_src", "copy_dst"):
        assert call(**{name: None}) == -1 and call(**{name: 0x9002}) == -1, name
    need = zf.lib().zf_compact_pages_workspace_size(100)
    assert need >= 400 and call(ws_bytes=need - 1) == -3
    assert zf.lib().zf_release_requests_workspace_size(-1) == 0 and zf.lib().zf_compact_pages_workspace_size(-1) == 0


def test_compaction_refuses_rows_that_32_bits_do_not_count(zf):
    """With the last few entries below 2^31 a row's pieces would be counted as negative, and its pages taken as unused."""
    f = zf.lib().zf_compact_pages
    for max_pages in ((1 << 30) + 1, 2 ** 31 - 256, 2 ** 31 - 255, 2 ** 31 - 1):
        assert f(1, max_pages, 100, 0x1000, 0x1100, 0x1200, 0x1300, 0x1400, 0x1500, 0x1600, None, 0x2000, 1 << 20, None) == -2


def test_copy_refuses(zf):
    f = zf.lib().zf_q4_copy_pages
    for kw, code in BAD_CACHES:
        assert f(ctypes.byref(_desc(zf, **kw)), 0x1000, 0x2000, 1, None) == code, kw
    d = ctypes.byref(_desc(zf))
    assert f(None, 0x1000, 0x2000, 1, None) == -1 and f(d, 0x1000, 0x2000, -1, None) == -1
    assert f(d, None, 0x2000, 1, None) == -1 and f(d, 0x1000, None, 1, None) == -1
    assert f(d, 0x1002, 0x2000, 1, None) == -1 and f(d, 0x1000, 0x2001, 1, None) == -1
    assert f(d, None, None, 0, None) == 0


def test_binding_refuses(zf):
    """Checks made on tensors, before the device is looked at; then the device itself."""
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    f32 = lambda *s: torch.zeros(s)  # noqa: E731
    cache = zf.Q4Cache(4, 2, 16, device="cpu")
    q, table, lens, start = torch.zeros(3, 8, 128, dtype=torch.bfloat16), i32(2, 4), i32(2), i32(3)
    ok = dict(q=q, page_table=table, seq_lens=lens, token_start=start)
    for kw, err in ((dict(q=q.float()), ValueError), (dict(q=q[..., :64]), ValueError), (dict(q=q[0]), ValueError),
                    (dict(q=[1]), TypeError), (dict(token_start=start.long()), ValueError), (dict(token_start=i32(3, 1)), ValueError),
                    (dict(token_start=i32(0)), ValueError), (dict(page_table=i32(1, 4)), ValueError),
                    (dict(seq_lens=i32(1)), ValueError), (dict(slopes=f32(7)), ValueError),
                    (dict(slopes=f32(8).double()), ValueError), (dict(out=torch.zeros(3, 8, 128)), ValueError),
                    (dict(out=torch.zeros(3, 128, 8, dtype=torch.bfloat16).transpose(1, 2)), ValueError),
                    (dict(lse=f32(8, 3)), ValueError), ({}, ValueError)):
        with pytest.raises(err):
            zf.q4_chunk_attn(cache, **{**ok, **kw})
    logits, u = f32(2, 50), f32(2)
    for args, kw, err in (((logits.double(), u), {}, ValueError), ((logits[0], u), {}, ValueError), ((logits, None), {}, ValueError),
                          ((logits, None), dict(tokens=i32(2), probs=f32(2, 50)), ValueError), ((logits, f32(3)), {}, ValueError),
                          ((logits, u), dict(temperature=f32(2).double()), ValueError), ((logits, u), dict(top_k=u), ValueError),
                          ((logits, u), dict(top_p=f32(1)), ValueError), ((logits, u), dict(min_p=i32(2)), ValueError),
                          ((logits, u), dict(probs=f32(2, 49)), ValueError), ((logits, u), dict(probs=f32(50, 2).t()), ValueError),
                          ((logits, u), dict(status=i32(2)), ValueError), ((logits, u), {}, ValueError)):
        with pytest.raises(err):
            zf.sample_tokens(*args, **kw)
    free, pos = i32(9), i32(1)
    fork = dict(page_table=table, seq_lens=lens, pages_held=lens, src=i32(1), dst=i32(1), free_pages=free, free_pos=pos, page_size=16)
    for kw in (dict(page_table=i32(2)), dict(page_table=i32(4, 2).t()), dict(seq_lens=i32(3)), dict(src=i32(1, 1)), dict(dst=i32(2)),
               dict(free_pages=i32(3, 3)), dict(free_pos=i32(2)), dict(src=u), {}):
        with pytest.raises(ValueError):
            zf.fork_requests(**{**fork, **kw})
    rel = dict(page_table=table, seq_lens=lens, pages_held=lens, release=lens, free_pages=free, free_pos=pos, num_pages=9)
    for kw in (dict(release=i32(3)), dict(free_pages=i32(18)[::2]), dict(pages_held=u), dict(page_table=lens), {}):
        with pytest.raises(ValueError):
            zf.release_requests(**{**rel, **kw})
    for kw in (dict(pages_held=i32(3)), dict(num_pages=-1), dict(page_table=lens), {}):
        with pytest.raises(ValueError):
            zf.compact_pages(**{**dict(page_table=table, pages_held=lens, num_pages=9), **kw})
    for s, d in ((i32(2), i32(3)), (i32(2, 1), i32(2)), (u, lens), (lens, lens)):
        with pytest.raises(ValueError):
            zf.q4_copy_pages(cache, s, d)


# ------------------------------------------------------------------------------ pins of the oracle
def test_chunk_oracle():
    rng = np.random.default_rng(3)
    k, v, q = rng.standard_normal((9, 2, 128)), rng.standard_normal((9, 2, 128)), rng.standard_normal((3, 4, 128))
    out, lse, *_ = R.chunk_attention(q, k, v, 6, 0.1, window=1)
    assert np.allclose(out, v[6:9].repeat(2, axis=1))                   # each row sees itself alone
    assert np.allclose(lse[0, 3], 0.1 * q[0, 3] @ k[6, 1])
    out, lse, *_ = R.chunk_attention(q, k * 0, v, -1, 0.1)
    assert not out[0].any() and np.isinf(lse[0]).all()                  # position -1 sees nothing
    assert np.allclose(out[2, 0], v[:2, 0].mean(0)) and np.allclose(lse[2], math.log(2))
    far = R.chunk_attention(q, k * 0, v, 6, 0.1, slopes=[50.0] * 4)[0]
    assert np.allclose(far, v[6:9].repeat(2, axis=1))                   # a steep slope: the nearest token
    low = R.chunk_attention(q, k * 100, v, 6, 1.0, softcap=1e-3)[1]
    assert np.allclose(low, np.log([7, 8, 9])[:, None], atol=2e-3)      # a low cap: all alike


def test_sampling_oracle():
    x = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
    p = lambda **kw: R.sample(x, **kw) / R.sample(x, **kw).sum()  # noqa: E731
    assert np.allclose(p(), [0.1, 0.4, 0.2, 0.3])
    assert np.allclose(p(top_k=2), [0, 4 / 7, 0, 3 / 7])
    assert np.allclose(p(top_p=0.69), [0, 4 / 7, 0, 3 / 7]) and np.allclose(p(top_p=0.71), [0, 4 / 9, 2 / 9, 3 / 9])
    assert np.allclose(p(min_p=0.6), [0, 4 / 7, 0, 3 / 7]) and np.allclose(p(top_k=3, top_p=0.7), [0, 4 / 7, 0, 3 / 7])
    assert np.allclose(p(temperature=0.0), [0, 1, 0, 0]) and np.allclose(p(temperature=0.5), np.array([1, 16, 4, 9]) / 30)
    assert np.allclose(R.sample(np.zeros(5), top_p=0.5) > 0, [1, 1, 1, 0, 0])
    assert R.sample(np.full(3, -np.inf)) is None and R.sample(x, min_p=1.5) is None
    assert R.draw(np.array([0, 4.0, 0, 3.0]), 0.0)[0] == 1 and R.draw(np.array([0, 4.0, 0, 3.0]), 0.999)[0] == 3


def test_page_oracle():
    table = np.array([[5, 2, 7, -1], [-1, -1, -1, -1], [-1, -1, -1, -1]])
    out = R.fork(table, [40, 0, 0], [3, 0, 0], [0, 0, 0], [1, 2, 1], [9, 8, 6], 0, 16)
    assert out[0].tolist() == [[5, 2, 7, -1], [5, 2, 9, -1], [5, 2, 8, -1]] and out[1:4] == ([40, 40, 40], [3, 3, 3], 2)
    assert out[4:] == ([7, 7, -1], [9, 8, -1], R.DEV_BAD_FORK)
    rel = R.release(out[0], out[1], out[2], [1, 1, 0], [0, 1, 3, 4, 6], 4, 10)
    assert rel == ([0, 0, 40], [0, 0, 3], [0, 1, 7, 9, 6], 2, 0)
    com = R.compact(out[0], rel[1], 10)
    assert com[0].tolist() == [[5, 2, 7, -1], [5, 2, 9, -1], [0, 2, 1, -1]] and com[2:] == (3, [5, 8, -1, -1, -1], [0, 1, -1, -1, -1], 0)
    assert com[1] == [-1, -1, -1, 3, 4, 5, 6, 7, 8, 9]
