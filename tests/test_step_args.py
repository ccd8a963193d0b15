"""The 4-bit cache, slot-map and draft-verification calls without a GPU: what they refuse before anything
is launched, in the C ABI and in the binding, and pins of their oracle."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import zf_step_oracle as S
from tests import helpers as H


@pytest.fixture(scope="module")
def zf():
    return H.zf_module()


def _desc(zf, **kw):
    d = dict(num_pages=4, num_kv_heads=2, head_dim=128, page_size=16, k_scale=1.0, v_scale=1.0, records=0x1000, status=None)
    d.update(kw)
    return zf.ZfQ4CacheDesc(**d)


BAD_CACHES = [(dict(head_dim=64), -1), (dict(page_size=8), -1), (dict(page_size=40), -1), (dict(page_size=144), -2),
              (dict(num_kv_heads=0), -1), (dict(num_pages=-1), -1), (dict(records=None), -1), (dict(records=0x1008), -1),
              (dict(k_scale=0.0), -1), (dict(k_scale=-1.0), -1), (dict(v_scale=float("nan")), -1),
              (dict(v_scale=float("inf")), -1), (dict(k_scale=1e-31), -1), (dict(v_scale=1e31), -1), (dict(status=0x1002), -1)]


@pytest.mark.parametrize("entry", ["zf_q4_write_tokens", "zf_q4_read_tokens"])
def test_token_calls_refuse(zf, entry):
    f = getattr(zf.lib(), entry)

    def call(desc, n=1, k=0x10000, v=0x20000, ids=0x30000, pos=0x40000):
        d = ctypes.byref(desc) if desc is not None else None
        return f(d, k, v, ids, pos, n, None) if "write" in entry else f(d, ids, pos, n, k, v, None)
    assert call(None) == -1
    for kw, code in BAD_CACHES:
        assert call(_desc(zf, **kw)) == code, kw
    d = _desc(zf)
    assert call(d, n=-1) == -1
    for name in ("k", "v", "ids", "pos"):
        assert call(d, **{name: None}) == -1
    assert call(d, k=0x10008) == -1 and call(d, v=0x20004) == -1 and call(d, ids=0x30002) == -1 and call(d, pos=0x40001) == -1
    assert call(_desc(zf, num_kv_heads=1 << 20), n=1 << 12) == -2          # more rows than the grid counts
    assert call(d, n=0) == 0


def test_attention_refuses(zf):
    f = zf.lib().zf_q4_decode_attn

    def call(desc, batch=2, tokens=1, hq=8, table=0x50000, max_pages=4, lens=0x60000, scale=0.1, q=0x10000, out=0x20000,
             lse=0x30000, ws=0x40000, ws_bytes=1 << 30):
        return f(ctypes.byref(desc), q, batch, tokens, hq, table, max_pages, lens, scale, out, lse, ws, ws_bytes, None)
    for kw, code in BAD_CACHES:
        assert call(_desc(zf, **kw)) == code, kw
    d = _desc(zf)
    for kw in (dict(batch=-1), dict(batch=4097), dict(tokens=0), dict(tokens=65), dict(hq=7), dict(hq=1), dict(max_pages=0),
               dict(q=None), dict(table=None), dict(lens=None), dict(out=None), dict(lse=None), dict(ws=None),
               dict(q=0x10004), dict(out=0x20008), dict(lse=0x30002), dict(ws=0x40004), dict(table=0x50001),
               dict(lens=0x60003), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=1e38),
               dict(max_pages=1 << 24)):
        assert call(d, **kw) == -1, kw
    assert call(_desc(zf, k_scale=1e30), scale=1e10) == -1                  # the scores' factor is no float
    assert call(_desc(zf, page_size=128, num_kv_heads=1), batch=4096, hq=1, max_pages=(1 << 16) + 1) == -2    # 2^31 records
    assert call(d, batch=0) == 0
    size = zf.lib().zf_q4_decode_attn_workspace_size
    for args in ((1, 0, 8, 2, 16, 4), (1, 1, 7, 2, 16, 4), (1, 1, 8, 2, 24, 4), (1, 1, 8, 2, 256, 4), (1, 1, 8, 2, 16, 0),
                 (4097, 1, 8, 2, 16, 4)):
        assert size(*args) == 0, args


def test_map_refuses(zf):
    f = zf.lib().zf_map_tokens
    names = ["batch", "page_size", "max_pages", "lens", "held", "new", "table", "free", "num_free", "pos", "out_lens",
             "out_held", "out_pos", "start", "ids", "positions", "seq", "max_tokens", "status", "stream"]
    good = [2, 16, 4, 0x1000, 0x1100, 0x1200, 0x2000, 0x3000, 8, 0x1300, 0x1400, 0x1500, 0x1600, 0x1700, 0x4000, 0x5000,
            0x6000, 10, None, None]

    def call(**kw):
        args = list(good)
        for k, v in kw.items():
            args[names.index(k)] = v
        return f(*args)
    for kw in (dict(batch=-1), dict(batch=4097), dict(page_size=0), dict(page_size=24), dict(max_pages=0),
               dict(max_pages=1 << 27), dict(num_free=-1), dict(max_tokens=-1), dict(max_tokens=(1 << 30) + 1), dict(ids=0x4004), dict(positions=0x5008),
               dict(seq=0x6002), dict(status=0x7001), dict(free=0x3002)):
        assert call(**kw) == -1, kw
    for name in ("lens", "held", "new", "table", "free", "pos", "out_lens", "out_held", "out_pos", "start", "ids",
                 "positions", "seq"):
        assert call(**{name: None}) == -1, name
        if name not in ("ids", "positions", "seq"):
            assert call(**{name: 0x9001}) == -1, name
    assert call(page_size=256) == -2
    assert call(batch=0, pos=None) == -1


def test_verify_refuses(zf):
    f = zf.lib().zf_verify_drafts
    names = ["batch", "drafts", "vocab", "target", "draft", "tokens", "n", "uniform", "accepted", "out", "lens", "new_lens",
             "status", "stream"]
    good = [2, 3, 100, 0x1000, 0x2000, 0x3000, 0x3100, 0x3200, 0x3300, 0x3400, None, None, None, None]

    def call(**kw):
        args = list(good)
        for k, v in kw.items():
            args[names.index(k)] = v
        return f(*args)
    for kw in (dict(batch=-1), dict(batch=4097), dict(drafts=0), dict(drafts=65), dict(vocab=0), dict(vocab=(1 << 24) + 1),
               dict(lens=0x4000), dict(new_lens=0x4000), dict(target=None), dict(tokens=None), dict(uniform=None),
               dict(accepted=None), dict(out=None), dict(target=0x1002), dict(draft=0x2001), dict(n=0x3102),
               dict(status=0x5001)):
        assert call(**kw) == -1, kw
    assert call(batch=0) == 0
    assert call(batch=0, lens=0x4000) == -1


def test_binding_checks_tokens_and_attention(zf):
    c = zf.Q4Cache(4, 2, 16, device="cpu")
    tok = torch.zeros(3, 2, 128, dtype=torch.int16)
    cases = [((tok[:2], tok, [0, 1, 2], [0, 0, 0]), "k_tok: shape"), ((tok, tok[..., :64], [0, 1, 2], [0, 0, 0]), "v_tok: shape"),
             ((tok.float(), tok, [0, 1, 2], [0, 0, 0]), "k_tok: dtype"), ((tok, tok.to("meta"), [0, 1, 2], [0, 0, 0]), "v_tok is on meta"),
             ((tok, tok, [0, 1, 2], [0, 0]), "positions: 2 entries"), ((tok, tok, [[0, 1, 2]], [0, 0, 0]), "page_ids: shape"),
             ((tok, tok, [0, 1, 2], [0, 0, 0]), "a CUDA device is needed")]
    for args, msg in cases:
        with pytest.raises(ValueError, match=msg):
            zf.q4_write_tokens(c, *args)
    with pytest.raises(ValueError, match="positions: 1 entries"):
        zf.q4_read_tokens(c, [0, 1], [0])
    with pytest.raises(ValueError, match="a CUDA device"):
        zf.q4_read_tokens(c, [0, 1], [0, 1])
    with pytest.raises(ValueError, match="records"):
        zf.Q4Cache(4, 2, 16, records=torch.zeros(4, 2, 1, 2303, dtype=torch.uint8))
    q, table, lens = torch.zeros(3, 8, 128, dtype=torch.int16), torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    cases = [((q.float(), table, lens), {}, "q: dtype"), ((q[..., :64], table, lens), {}, "q: shape"),
             ((q[0], table, lens), {}, "q: shape"), ((q, table.long(), lens), {}, "page_table: dtype"),
             ((q, table[0], lens), {}, "page_table: shape"), ((q, table[:2], lens), {}, "page_table: 2 rows"),
             ((q, table, lens[:2]), {}, "seq_lens: 2 rows"), ((q, table, lens.to("meta")), {}, "seq_lens is on meta"),
             ((q, table, lens), dict(out=torch.zeros(3, 8, 64)), "out: shape"),
             ((q, table, lens), dict(out=torch.zeros(3, 128, 8).transpose(1, 2)), "out must be contiguous"),
             ((q, table, lens), dict(lse=torch.zeros(3, 8, dtype=torch.float64)), "lse: dtype"),
             ((q, table, lens), dict(workspace=torch.zeros(8, 8).t()), "workspace must be contiguous"),
             ((q, table, lens), dict(workspace=torch.zeros(8, device="meta")), "workspace is on meta"),
             ((q, table, lens), {}, "a CUDA device")]
    for args, kw, msg in cases:
        with pytest.raises(ValueError, match=msg):
            zf.q4_decode_attn(c, *args, **kw)
    with pytest.raises(TypeError):
        zf.q4_decode_attn(c, q.numpy(), table, lens)


def test_binding_checks_map_and_verify(zf):
    def i(*shape):
        return torch.zeros(shape, dtype=torch.int32)
    good = [i(3, 4), i(3), i(3), i(3), i(9), i(1)]
    bad = [(0, i(3), "page_table must be"), (0, i(4, 3).t(), "page_table must be contiguous"), (1, i(2), "seq_lens: shape"),
           (2, i(3).long(), "pages_held: dtype"), (3, i(3).to("meta"), "new_tokens is on meta"), (4, i(3, 3), "free_pages must be"),
           (5, i(2), "free_pos: shape")]
    for at, x, msg in bad:
        args = list(good)
        args[at] = x
        with pytest.raises(ValueError, match=msg):
            zf.map_tokens(*args, 16, 5)
    out = zf.TokenMap(i(3), i(3), i(1), i(3), i(5), i(5), i(5))
    with pytest.raises(ValueError, match="out.token_start: shape"):
        zf.map_tokens(*good, 16, 5, out=out)
    with pytest.raises(ValueError, match="status: shape"):
        zf.map_tokens(*good, 16, 5, status=i(2))
    with pytest.raises(ValueError, match="a CUDA device"):
        zf.map_tokens(*good, 16, 5)
    p, q, d, u = torch.zeros(2, 4, 9), torch.zeros(2, 3, 9), i(2, 3), torch.zeros(2, 4)
    cases = [((p, i(6), u), {}, "draft_tokens must be"), ((p[0], d, u), {}, "target_probs must be"),
             ((p[:, :3], d, u), {}, "target_probs: shape"), ((p.double(), d, u), {}, "target_probs: dtype"),
             ((p, d.long(), u), {}, "draft_tokens: dtype"), ((p, d, u[:, :3]), {}, "uniform: shape"),
             ((p, d, u), dict(draft_probs=p), "draft_probs: shape"), ((p, d, u), dict(n_drafts=i(3)), "n_drafts: shape"),
             ((p, d, u), dict(seq_lens=i(2)), "go together"), ((p, d, u), dict(new_seq_lens=i(2)), "go together"),
             ((p, d, u), dict(seq_lens=i(2), new_seq_lens=i(4)[::2]), "new_seq_lens must be contiguous"),
             ((p, d, u), dict(status=i(1, 1)), "status: shape"), ((p, d, u), {}, "a CUDA device")]
    for args, kw, msg in cases:
        with pytest.raises(ValueError, match=msg):
            zf.verify_drafts(*args, **kw)


# ------------------------------------------------------------------------------------ oracle pins
def test_oracle_number_formats():
    assert S.E4M3[0] == 0 and S.E4M3[1] == 2.0 ** -9 and S.E4M3[8] == 2.0 ** -6 and S.E4M3[126] == 448
    assert (np.diff(S.E4M3) > 0).all()
    assert torch.equal(torch.tensor(S.E4M3, dtype=torch.float32), torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float())
    x = np.linspace(0, 480, 5000)
    want = torch.tensor(x, dtype=torch.float32).clamp(max=448).to(torch.float8_e4m3fn).float().numpy()
    assert [S.E4M3[S.nearest_even(S.E4M3, float(np.float32(v)))] for v in x] == want.tolist()
    for lo, hi, even in ((0, 1, 0), (1, 2, 2), (2, 3, 2), (3, 4, 4), (4, 5, 4), (5, 6, 6), (6, 7, 6)):
        assert S.nearest_even(S.E2M1, (S.E2M1[lo] + S.E2M1[hi]) / 2) == even
    assert S.nearest_even(S.E2M1, 100.0) == 7


def test_oracle_layout_covers_the_record():
    at = [S.k_code_at(t, b) for t in range(16) for b in range(64)] + [S.v_code_at(t, b) for t in range(16) for b in range(64)]
    at += [S.k_scale_at(t, c) for t in range(16) for c in range(8)] + [S.v_scale_at(t, c) for t in range(16) for c in range(8)]
    assert sorted(at) == list(range(S.RECORD))


def test_oracle_quantisation_error():
    """A stored value is off by at most the block's scale: half the widest gap between codes (6 - 4); a scale
    that was rounded down by its half step (1/16 of 6) saturates within 0.4 of it."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((40, 16)).astype(np.float32)
    for row in x:
        bits = S.f64_to_bf16(row.astype(np.float64))
        codes, byte, odd = S.quantise_block(bits)
        got = S.E2M1[codes & 7] * np.where(codes > 7, -1, 1) * S.E4M3[byte]
        assert not odd and (np.abs(got - S.bf16_to_f64(bits)) <= 1.0 * S.E4M3[byte] * (1 + 1e-12)).all()
    codes, byte, _ = S.quantise_block(np.zeros(16, np.uint16))
    assert byte == 0 and not codes.any()


def test_oracle_map_and_verify_pins():
    table, lens, held, pos, start, ids, positions, seq, st = S.map_tokens(
        [[5, -1, -1], [7, 8, -1]], [15, 17], [1, 2], [2, 0], [9, 3], 0, 16, 4)
    assert table == [[5, 9, -1], [7, 8, -1]] and lens == [17, 17] and held == [2, 2] and pos == 1
    assert start == [0, 2, 2] and ids == [5, 9, -1, -1] and positions == [15, 0, -1, -1] and seq == [15, 16, -1, -1] and st == 0
    # a request that was shortened uses the page it kept
    out = S.map_tokens([[5, 6]], [10], [2], [10], [], 0, 16, 10)
    assert out[0] == [[5, 6]] and out[5] == [5] * 6 + [6] * 4 and out[3] == 0
    p = np.array([[[0.5, 0.5, 0.0], [0.1, 0.2, 0.7]]], np.float32)
    q = np.array([[[0.25, 0.75, 0.0]]], np.float32)
    for u, acc, tok in ((0.6, 1, [1, 2]), (0.7, 0, [0, -1])):       # 0.5 / 0.75 = 0.667 is the border
        a, t, _, _ = S.verify(p, q, np.array([[1]]), None, np.array([[u, 0.9]], np.float32))
        assert a == [acc] and t == [tok]
