"""The 4-bit cache on the GPU: stored bytes against the oracle's, values read back, and attention over it
against the float64 oracle with a bound from the number of roundings."""
import math

import numpy as np
import pytest
import torch

from oracle import zf_step_oracle as S
from tests import helpers as H

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zf():
    return H.zf_module()


def bits(x):
    return torch.as_tensor(x).to(torch.bfloat16).view(torch.int16)


def tokens(n, hkv, seed, spread=0.5):
    """K with per-channel spread and strong channels, V normal; some blocks of zeros and tiny values."""
    rng = np.random.default_rng(seed)
    s = np.exp(spread * rng.standard_normal(128))
    s[:4] *= 10
    k = rng.standard_normal((n, hkv, 128)) * s
    v = rng.standard_normal((n, hkv, 128))
    v[rng.random((n, hkv)) < 0.05] = 0
    v[..., 32:48] *= 1e-3
    return bits(k.astype(np.float32)), bits(v.astype(np.float32))


def place(n, pool, page, seed):
    """n distinct (page, position) places."""
    at = np.random.default_rng(seed).permutation(pool * page)[:n]
    return (at // page).tolist(), (at % page).tolist()


@pytest.mark.parametrize("page,hkv,n", [(16, 1, 1), (16, 8, 33), (48, 3, 70), (128, 2, 200)])
@pytest.mark.parametrize("scales", [(1.0, 1.0), (0.37, 5.0)])
def test_written_bytes_match_the_oracle(zf, page, hkv, n, scales):
    pool = -(-n // page) + 2
    k, v = tokens(n, hkv, 1000 + n)
    ids, pos = place(n, pool, page, n)
    c = zf.Q4Cache(pool, hkv, page, k_scale=scales[0], v_scale=scales[1])
    zf.q4_write_tokens(c, k.cuda(), v.cuda(), ids, pos)
    o = S.Q4Cache(pool, hkv, page, *scales)
    o.write(H.np_bits(k), H.np_bits(v), ids, pos)
    assert (c.records.cpu().numpy() == o.records).all()
    assert c.status_word() == o.status == 0
    kr, vr = zf.q4_read_tokens(c, ids, pos)
    for i in range(n):
        for h in range(hkv):
            ek, ev = o.token(ids[i], h, pos[i])
            # float32 product of the stored value (exact) and the cache's scale, then one rounding to BF16:
            # exact for scale 1, else within half a step of either (2^-8 + 2^-24)
            tol = 0 if scales == (1.0, 1.0) else 2.0 ** -8 + 2.0 ** -23
            for got, want in ((kr, ek), (vr, ev)):
                x = S.bf16_to_f64(H.np_bits(got[i, h]))
                assert (np.abs(x - want) <= tol * np.abs(want)).all()


def test_borders_between_codes_and_scales(zf):
    """Every quotient that lies exactly between two codes, for every scale; every maximum between two scales."""
    rows = []
    for byte in range(1, 127):
        s = S.E4M3[byte]
        row = [6 * s] + [b * s for b in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)] + [-0.0]
        row += [-b * s for b in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)]
        rows.append(row)
    for byte in range(126):
        mid = (S.E4M3[byte] + S.E4M3[byte + 1]) / 2
        rows.append([6 * mid, -6 * mid] + [6 * mid * f for f in np.linspace(-1, 1, 14)])
    rows += [[0.0] * 16, [-0.0] * 16, [1e-30] * 16, [3e38, -3e38] + [1.0] * 14, [2688.0] * 8 + [2690.0] * 8]
    while len(rows) % 8:
        rows.append([1.0] * 16)
    x = bits(np.array(rows, np.float32).reshape(-1, 1, 128))
    n = x.shape[0]
    c = zf.Q4Cache(4, 1, 16)
    o = S.Q4Cache(4, 1, 16)
    ids, pos = [i // 16 for i in range(n)], [i % 16 for i in range(n)]
    flip = x.flip(0).contiguous()
    zf.q4_write_tokens(c, x.cuda(), flip.cuda(), ids, pos)
    o.write(H.np_bits(x), H.np_bits(flip), ids, pos)
    got = c.records.cpu().numpy()
    assert (got == o.records).all(), [(i.tolist(), got[tuple(i)], o.records[tuple(i)]) for i in np.argwhere(got != o.records)[:8]]


def test_values_that_are_not_finite(zf):
    x = torch.randn(3, 2, 128)
    x[0, 0, 5] = math.nan
    x[1, 1, 20] = math.inf
    x[1, 1, 100] = -math.inf
    k, v = bits(x), bits(torch.randn(3, 2, 128))
    c, o = zf.Q4Cache(1, 2, 16), S.Q4Cache(1, 2, 16)
    zf.q4_write_tokens(c, k.cuda(), v.cuda(), [0, 0, 0], [3, 4, 5])
    o.write(H.np_bits(k), H.np_bits(v), [0, 0, 0], [3, 4, 5])
    assert (c.records.cpu().numpy() == o.records).all()
    assert c.status_word() == o.status == zf.DEV_NOT_FINITE
    kr, _ = zf.q4_read_tokens(c, [0, 0], [3, 4])
    kr = kr.view(torch.bfloat16)
    assert kr.isfinite().all() and kr[0, 0, 5] == 0 and kr[1, 1, 20] == 2688 and kr[1, 1, 100] == -2688


def test_bad_and_skipped_entries(zf):
    k, v = tokens(5, 2, 7)
    c = zf.Q4Cache(2, 2, 16)
    before = torch.randint(0, 120, c.records.shape, dtype=torch.uint8, device="cuda")
    c.records.copy_(before)
    zf.q4_write_tokens(c, k.cuda(), v.cuda(), [0, 5, -1, 0, 7], [-1, -1, -1, -1, -1])
    assert torch.equal(c.records, before) and c.status_word() == 0
    zf.q4_write_tokens(c, k.cuda(), v.cuda(), [2, -1, 1, 0, 0], [0, 3, 16, -2, -1])
    assert torch.equal(c.records, before)
    assert c.status_word() == zf.DEV_BAD_PAGE_ID | zf.DEV_BAD_N_VALID
    kr, vr = zf.q4_read_tokens(c, [2, 0], [0, -1])
    assert not kr.any() and not vr.any()
    zf.q4_write_tokens(c, k[:0].cuda(), v[:0].cuda(), [], [])


CASES = [
    # batch lens, hkv, group, T, page
    ([1], 1, 1, 1, 16),
    ([0, 1, 15, 16, 17, 31, 32, 33, 300], 2, 4, 1, 16),
    ([130, 0, 64], 1, 7, 1, 64),
    ([97, 1, 200], 3, 2, 4, 48),             # 8 columns, causal, a request shorter than T
    ([97, 3, 0, 130], 1, 8, 2, 16),          # 16 columns
    ([70, 129], 2, 5, 2, 32),                # 10 columns of 16
    ([257, 2], 1, 7, 4, 128),                # 28 columns of 32
    ([150, 40], 1, 8, 5, 16),                # 40 columns: two passes of 24
    ([65], 1, 3, 8, 16),                     # 24 columns
    ([90], 1, 1, 64, 16),                    # 64 new tokens
    ([900, 1200], 2, 4, 1, 16),              # several partials per request
    ([900, 0, 1203], 2, 4, 5, 16),           # 20 columns of 24, the same
    ([131, 18], 1, 11, 3, 16),               # 33 columns: two passes of 24
    ([100, 9], 1, 9, 9, 48),                 # 81 columns: three passes of 32
    ([600, 40], 1, 16, 4, 16),               # 64 columns: two passes of 32
]


def build(zf, lens, hkv, page, seed, k_scale=1.0, v_scale=1.0):
    pages = [-(-L // page) for L in lens]
    pool = sum(pages) + 2
    perm = np.random.default_rng(seed).permutation(pool)
    table = np.full((len(lens), max(max(pages), 1) + 1), -1, np.int32)
    ids, pos, at = [], [], 0
    for b, L in enumerate(lens):
        table[b, :pages[b]] = perm[at:at + pages[b]]
        at += pages[b]
        ids += [int(table[b, p // page]) for p in range(L)]
        pos += [p % page for p in range(L)]
    k, v = tokens(max(len(ids), 1), hkv, seed + 1)
    k, v = k[:len(ids)], v[:len(ids)]
    c, o = zf.Q4Cache(pool, hkv, page, k_scale=k_scale, v_scale=v_scale), S.Q4Cache(pool, hkv, page, k_scale, v_scale)
    # what lies past the contexts may be anything
    g = torch.Generator().manual_seed(seed)
    c.records.copy_(torch.randint(0, 256, c.records.shape, dtype=torch.uint8, generator=g))
    zf.q4_write_tokens(c, k.cuda(), v.cuda(), ids, pos)
    o.records[...] = c.records.cpu().numpy()       # (bytes are compared in the tests above)
    return c, o, torch.from_numpy(table), torch.tensor(lens, dtype=torch.int32)


def check(out, lse, ref, ref_lse, bound, vmax, lse_tol):
    out, lse = out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    empty = np.isneginf(ref_lse)
    assert (np.isneginf(lse) == empty).all() and (out[empty] == 0).all()
    off = np.abs(out - ref).max(-1)
    assert (off <= bound * vmax)[~empty].all(), (off / np.maximum(bound * vmax, 1e-300)).max()
    if (~empty).any():
        d = np.abs(lse[~empty] - ref_lse[~empty])
        assert (d <= lse_tol[~empty] + 2.0 ** -22 * np.abs(ref_lse[~empty])).all(), d.max()


@pytest.mark.parametrize("lens,hkv,group,T,page", CASES)
def test_attention_matches_the_oracle(zf, lens, hkv, group, T, page):
    c, o, table, sl = build(zf, lens, hkv, page, 10 * len(lens) + T)
    q = bits(torch.randn(len(lens), T, hkv * group, 128, generator=torch.Generator().manual_seed(5)))
    scale = 1 / math.sqrt(128)
    out, lse = zf.q4_decode_attn(c, q.cuda(), table.cuda(), sl.cuda())
    ref, ref_lse, bound = S.attention(o, H.np_bits(q), table.numpy(), lens, scale)
    check(out, lse, ref, ref_lse, bound, 20.0 * 1.0 if not lens else 6.0, bound)
    assert c.status_word() == 0
    if T == 1:      # the three-dimensional form is the same call
        o3, l3 = zf.q4_decode_attn(c, q[:, 0].cuda(), table.cuda(), sl.cuda())
        assert torch.equal(o3, out[:, 0]) and torch.equal(l3, lse[:, 0])
    again = zf.q4_decode_attn(c, q.cuda(), table.cuda(), sl.cuda())
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


def test_the_largest_calls_workspace_serves_smaller_ones(zf):
    for hq, hkv in [(32, 8), (28, 4), (11, 1)]:
        def size(batch, T, pages):
            return zf.q4_workspace_size(batch, T, hq, hkv, 16, pages)
        by_tokens = [size(8, T, 64) for T in range(1, 33)]
        assert by_tokens[0] > 0 and by_tokens == sorted(by_tokens)
        by_batch = [size(b, 5, 3) for b in range(1, 40)]
        assert by_batch == sorted(by_batch)
        by_pages = [size(2, 3, p) for p in range(1, 40)]
        assert by_pages == sorted(by_pages)
    c, _, table, sl = build(zf, [40, 75], 1, 16, 3)
    q = bits(torch.randn(2, 3, 11, 128, generator=torch.Generator().manual_seed(6))).cuda()
    ws = torch.empty(zf.q4_workspace_size(2, 9, 11, 1, 16, table.shape[1]), dtype=torch.uint8, device="cuda")
    for T in (1, 2, 3):
        want = zf.q4_decode_attn(c, q[:, :T].contiguous(), table.cuda(), sl.cuda())
        got = zf.q4_decode_attn(c, q[:, :T].contiguous(), table.cuda(), sl.cuda(), workspace=ws)
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("k_scale,v_scale,scale", [(0.25, 3.0, 0.05), (1.0, 1.0, -0.08), (1.0, 1.0, 0.0)])
def test_cache_scales_and_softmax_scales(zf, k_scale, v_scale, scale):
    c, o, table, sl = build(zf, [77, 20], 2, 16, 3, k_scale, v_scale)
    q = bits(torch.randn(2, 1, 6, 128, generator=torch.Generator().manual_seed(6)))
    out, lse = zf.q4_decode_attn(c, q.cuda(), table.cuda(), sl.cuda(), scale)
    ref, ref_lse, bound = S.attention(o, H.np_bits(q), table.numpy(), [77, 20], scale)
    check(out, lse, ref, ref_lse, bound, 8.0, bound)


def test_query_magnitudes(zf):
    """Rows of very large and very small queries, zeros, and rows with a NaN or an infinity, which stay alone."""
    c, o, table, sl = build(zf, [100], 1, 16, 4)
    q = torch.randn(1, 1, 8, 128, generator=torch.Generator().manual_seed(7))
    q[0, 0, 0] *= 1e30
    q[0, 0, 1] *= 1e-30
    q[0, 0, 2] = 0
    q[0, 0, 3] *= torch.logspace(-6, 0, 128)
    q[0, 0, 4, 9] = math.nan
    q[0, 0, 5, 9] = math.inf
    q = bits(q)
    out, lse = zf.q4_decode_attn(c, q.cuda(), table.cuda(), sl.cuda(), 1e-31)
    assert out[0, 0, 4].isnan().all() and lse[0, 0, 4].isnan()
    assert out[0, 0, 5].isnan().all()
    keep = [0, 1, 2, 3, 6, 7]
    ref, ref_lse, bound = S.attention(o, H.np_bits(q[:, :, keep]), table.numpy(), [100], 1e-31)
    # the largest row's weights meet scores around 1; one fp16 rounding of 2^-36 of the row's maximum is below the bound
    o.hkv = 1
    check(out[:, :, keep], lse[:, :, keep], ref, ref_lse, bound, 6.0, bound)


@pytest.mark.parametrize("power", [20, 40, 90])
def test_scores_beyond_float_steps_of_one(zf, power):
    """Scores so large that neighbouring floats lie further apart than any exponent: the largest score takes
    all the weight, over one unit, several units and several ranges."""
    for lens in ([31], [700], [5000]):
        c, o, table, sl = build(zf, lens, 1, 16, 30 + power)
        q = torch.randn(1, 1, 8, 128, generator=torch.Generator().manual_seed(9)) * 2.0 ** power
        kv = [o.token(int(table[0, p // 16]), 0, p % 16) for p in range(lens[0])]
        k, v = np.array([x[0] for x in kv]), np.array([x[1] for x in kv])
        q = bits(q)
        out, lse = zf.q4_decode_attn(c, q.cuda(), table.cuda(), sl.cuda(), 1.0)
        s = k @ S.bf16_to_f64(H.np_bits(q[0, 0])).T
        order = np.sort(s, 0)
        clear = order[-1] - order[-2] > 1e-4 * np.abs(s).max(0)           # above any rounding of the scores
        assert clear.any() and torch.isfinite(out).all() and torch.isfinite(lse).all()
        got = out[0, 0].cpu().numpy()
        for g in np.nonzero(clear)[0]:
            # one weight of 1: the value itself, up to the split's and the division's rounding
            assert (np.abs(got[g] - v[s[:, g].argmax()]) <= 2.0 ** -21 * np.abs(v).max()).all()


def test_nan_row_with_partials(zf):
    """A NaN query row over a context that is split: the merge keeps the NaN, the other rows their values."""
    c, o, table, sl = build(zf, [5000], 1, 16, 8)
    q = torch.randn(1, 1, 2, 128, generator=torch.Generator().manual_seed(9))
    q[0, 0, 1] = math.nan
    q = bits(q)
    out, lse = zf.q4_decode_attn(c, q.cuda(), table.cuda(), sl.cuda())
    assert out[0, 0, 1].isnan().all() and lse[0, 0, 1].isnan()
    ref, ref_lse, bound = S.attention(o, H.np_bits(q[:, :, :1]), table.numpy(), [5000], 1 / math.sqrt(128))
    check(out[:, :, :1], lse[:, :, :1], ref, ref_lse, bound, 6.0, bound)


def test_bad_pages_and_lengths(zf):
    c, o, table, sl = build(zf, [100, 60], 1, 16, 11)
    table[0, 2] = 1000
    table[1, 0] = -1
    q = bits(torch.randn(2, 1, 4, 128, generator=torch.Generator().manual_seed(8)))
    out, lse = zf.q4_decode_attn(c, q.cuda(), table.cuda(), sl.cuda())
    assert c.status_word() == zf.DEV_BAD_PAGE_ID
    ref, ref_lse, bound = S.attention(o, H.np_bits(q), table.numpy(), [100, 60], 1 / math.sqrt(128))
    check(out, lse, ref, ref_lse, bound, 6.0, bound)
    c.status.zero_()
    over = sl.clone()
    over[1] = -5
    zf.q4_decode_attn(c, q.cuda(), table.cuda(), over.cuda())
    assert c.status_word() & zf.DEV_BAD_SEQ_LEN


def test_workspace_too_small_is_refused(zf):
    c, o, table, sl = build(zf, [100], 1, 16, 12)
    q = bits(torch.randn(1, 4, 128)).cuda()
    with pytest.raises(zf.ZfError, match="workspace too small"):
        zf.q4_decode_attn(c, q, table.cuda(), sl.cuda(), workspace=torch.empty(128, dtype=torch.uint8, device="cuda"))


def test_another_stream_and_a_captured_graph(zf):
    """The same results on a side stream and from a graph replayed with other lengths; rows of idle requests."""
    lens = [500, 33, 0, 220]
    c, o, table, sl = build(zf, lens, 2, 16, 13)
    q = bits(torch.randn(4, 2, 8, 128, generator=torch.Generator().manual_seed(8))).cuda()
    tab, sl = table.cuda(), sl.cuda()
    want = zf.q4_decode_attn(c, q, tab, sl)
    shorter = (sl - 3).clamp(min=0)
    want2 = zf.q4_decode_attn(c, q, tab, shorter)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = zf.q4_decode_attn(c, q, tab, sl)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    ws = zf.new_workspace(zf.q4_workspace_size(4, 2, 8, 2, 16, tab.shape[1]))
    live = sl.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = zf.q4_decode_attn(c, q, tab, live, workspace=ws)
    for lens_now, ref in ((sl, want), (shorter, want2), (sl, want)):
        live.copy_(lens_now)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])


def test_stream_argument_orders_the_whole_call(zf):
    """stream=: inputs that have to be converted, outputs and workspace live on that stream, behind a slow writer."""
    lens = [300, 77]
    c, o, table, sl = build(zf, lens, 2, 16, 15)
    k, v = tokens(6, 2, 99)
    ids, pos = [int(table[0, 0])] * 6, list(range(6))
    q = bits(torch.randn(2, 1, 8, 128, generator=torch.Generator().manual_seed(8)))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        kd = torch.zeros(6, 128, 2, dtype=torch.int16, device="cuda")
        torch.cuda._sleep(20_000_000)
        kd.copy_(k.transpose(1, 2))                       # a strided source, written late on s
        vd = v.cuda()
    zf.q4_write_tokens(c, kd.transpose(1, 2), vd, ids, pos, stream=s)
    kr, vr = zf.q4_read_tokens(c, ids, pos, stream=s)
    with torch.cuda.stream(s):
        qd, td, sd = q.cuda(), table.cuda(), sl.cuda()
    out, lse = zf.q4_decode_attn(c, qd, td, sd, stream=s)
    s.synchronize()
    w = S.Q4Cache(c.num_pages, 2, 16)
    w.records[...] = o.records
    w.write(H.np_bits(k), H.np_bits(v), ids, pos)
    assert (c.records.cpu().numpy() == w.records).all()
    assert (S.bf16_to_f64(H.np_bits(kr[3, 1])) == w.token(ids[3], 1, pos[3])[0]).all()
    ref, ref_lse, bound = S.attention(w, H.np_bits(q), table.numpy(), lens, 1 / math.sqrt(128))
    check(out, lse, ref, ref_lse, bound, 6.0, bound)


def test_two_calls_at_once(zf):
    """Calls on two streams with workspaces of their own."""
    runs = []
    for seed, lens in ((16, [900, 40]), (17, [33, 700, 5])):
        c, o, table, sl = build(zf, lens, 2, 16, seed)
        q = bits(torch.randn(len(lens), 2, 8, 128, generator=torch.Generator().manual_seed(seed)))
        runs.append((c, q.cuda(), table.cuda(), sl.cuda()))
    want = [zf.q4_decode_attn(*r) for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    got = []
    for _ in range(5):
        got += [(i, zf.q4_decode_attn(*r, stream=s)) for i, (r, s) in enumerate(zip(runs, streams))]
    torch.cuda.synchronize()
    for i, (out, lse) in got:
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


def test_cache_beyond_4_gib(zf):
    """Records whose byte offsets pass 32 bits: written, read back and attended on a cache's last pages."""
    page, hkv, lens = 128, 8, [200, 130]
    pages = 31000
    c = zf.Q4Cache(pages, hkv, page)
    assert c.stored_bytes() > 1 << 32
    small = S.Q4Cache(4, hkv, page)
    at = [pages - 1, 5, pages - 2, pages // 2]               # page i of the small cache
    ids = [0] * 128 + [1] * 72 + [2] * 128 + [3] * 2
    pos = list(range(128)) + list(range(72)) + list(range(128)) + [0, 1]
    k, v = tokens(len(ids), hkv, 18)
    big = [at[i] for i in ids]
    zf.q4_write_tokens(c, k.cuda(), v.cuda(), big, pos)
    small.write(H.np_bits(k), H.np_bits(v), ids, pos)
    for i, p in enumerate(at):
        assert (c.records[p].cpu().numpy() == small.records[i]).all()
    kr, _ = zf.q4_read_tokens(c, big, pos)
    assert (S.bf16_to_f64(H.np_bits(kr[0, 7])) == small.token(0, 7, 0)[0]).all()
    q = bits(torch.randn(2, 8, 128, generator=torch.Generator().manual_seed(19)))
    out, lse = zf.q4_decode_attn(c, q.cuda(), i32([at[:2], at[2:]]).cuda(), i32(lens).cuda())
    ref, ref_lse, bound = S.attention(small, H.np_bits(q)[:, None], np.array([[0, 1], [2, 3]]), lens, 1 / math.sqrt(128))
    check(out[:, None], lse[:, None], ref, ref_lse, bound, 6.0, bound)


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def test_many_requests_and_an_empty_batch(zf):
    """4096 requests of zero to three records (ranges that end inside pairs, pairs without records), and none."""
    rng = np.random.default_rng(20)
    lens = rng.integers(0, 40, 4096).tolist()
    c, o, table, sl = build(zf, lens, 1, 16, 21)
    q = bits(torch.randn(4096, 1, 2, 128, generator=torch.Generator().manual_seed(22)))
    out, lse = zf.q4_decode_attn(c, q.cuda(), table.cuda(), sl.cuda())
    pick = rng.permutation(4096)[:300]
    ref, ref_lse, bound = S.attention(o, H.np_bits(q)[pick], table.numpy()[pick], [lens[i] for i in pick], 1 / math.sqrt(128))
    check(out[pick.tolist()], lse[pick.tolist()], ref, ref_lse, bound, 6.0, bound)
    o0, l0 = zf.q4_decode_attn(c, q[:0].cuda(), table.cuda(), sl.cuda())
    assert o0.shape == (0, 1, 2, 128) and l0.shape == (0, 1, 2)
