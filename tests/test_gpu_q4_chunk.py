"""Attention of a ragged batch of new tokens over the 4-bit cache, against the float64 oracle with bounds from the
number of roundings."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import zf_serve_oracle as R
from oracle import zf_step_oracle as S
from tests import helpers as H
from tests.test_step_args import _desc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zf():
    return H.zf_module()


def f64(x):
    return S.bf16_to_f64(H.np_bits(x.view(torch.int16)))


class Case:
    """Requests of given lengths and new tokens over a shuffled pool; keys with strong channels."""

    def __init__(self, zf, page, hkv, group, lens, new, seed=0, scales=(1.0, 1.0), lead=0, behind=0, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        self.hkv, self.hq, self.page, self.lens, self.new, self.lead = hkv, hkv * group, page, lens, new, lead
        count = [-(-L // page) for L in lens]
        pool, max_pages = sum(count) + 2, max(count + [1])
        perm = torch.randperm(pool, generator=g).tolist()
        table, at = np.full((len(lens), max_pages), -1, np.int32), 0
        for b, c in enumerate(count):
            table[b, :c] = perm[at:at + c]
            at += c
        self.table = torch.from_numpy(table)
        self.cache = zf.Q4Cache(pool, hkv, page, k_scale=scales[0], v_scale=scales[1])
        self.k, self.v = [], []
        s = torch.ones(128) * spread
        s[:4] *= 8
        for b, L in enumerate(lens):
            k = (torch.randn(L, hkv, 128, generator=g) * s * scales[0]).to(torch.bfloat16)
            v = (torch.randn(L, hkv, 128, generator=g) * scales[1]).to(torch.bfloat16)
            ids = [int(table[b, p // page]) for p in range(L)]
            pos = [p % page for p in range(L)]
            zf.q4_write_tokens(self.cache, k.cuda(), v.cuda(), ids, pos)
            raw = zf.Q4Cache(pool, hkv, page, records=self.cache.records)            # scale 1: exact in BF16
            rk, rv = zf.q4_read_tokens(raw, ids, pos)
            self.k.append(f64(rk) * np.float32(scales[0]).astype(np.float64))
            self.v.append(f64(rv) * np.float32(scales[1]).astype(np.float64))
        self.start = np.cumsum([lead] + list(new)).astype(np.int32)
        self.rows = int(self.start[-1]) + behind
        self.q = torch.randn(self.rows, self.hq, 128, generator=g).to(torch.bfloat16)

    def args(self):
        return (self.cache, self.q.cuda(), self.table.cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda(),
                torch.from_numpy(self.start).cuda())

    def check(self, out, lse, scale=None, window=0, softcap=0.0, slopes=None, requests=None, seen=None):
        scale = 1 / math.sqrt(128) if scale is None else scale
        out, lse = f64(out), lse.double().cpu().numpy()
        for b in range(len(self.lens)) if requests is None else requests:
            a, e = self.start[b], self.start[b + 1]
            want, wl, wv, sv, mag = R.chunk_attention(f64(self.q[a:e]), self.k[b], self.v[b], self.lens[b] - self.new[b],
                                                      scale, window, softcap, slopes, None if seen is None else seen[b])
            # a score: up to 128 additions of products, each off by 2^-23 of their magnitudes' sum (the tensor core
            # truncates), a few roundings more, in log2 units and back; the cap's tanh; the slopes' products
            far = 0 if slopes is None else np.abs(slopes).max() * min(self.lens[b], window or self.lens[b])
            off = mag * 2.0 ** -16 + 2.0 ** -20 + softcap * 2.0 ** -20 + far * 2.0 ** -22
            # weights: fp16 (2^-11, or 2^-32 of the row's largest) and a score's error twice (numerator, sum)
            tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2 * off + 2.0 ** -18)[..., None] * wv + 2.0 ** -32 * sv + 1e-30
            assert (np.abs(out[a:e] - want) <= tol).all(), (b, np.abs(out[a:e] - want).max(), (np.abs(out[a:e] - want) / tol).max())
            none = np.isinf(wl)
            assert (lse[a:e][none] == -np.inf).all() and not out[a:e][none].any()
            assert (np.abs(lse[a:e][~none] - wl[~none]) <= off[~none] + 2.0 ** -20 * (1 + np.abs(wl[~none]))).all()


SHAPES = [
    (16, 1, 1, [1], [1]),                                            # one token over itself
    (16, 2, 4, [200, 37, 0, 129, 16], [64, 37, 0, 1, 16]),           # a last tile of every kind
    (48, 1, 7, [127, 128, 129, 255, 256, 257], [127, 1, 3, 36, 37, 19]),   # rows 889, 7, 21, 252, 259, 133
    (64, 2, 8, [300, 16], [16, 16]),                                 # exactly 128 rows
    (32, 1, 3, [500, 90], [86, 43]),                                 # 258 and 129 rows
    (128, 3, 5, [700], [13]),
    (16, 1, 300, [40], [2]),                                         # one token's rows span units
    (16, 4, 2, [5, 3, 140], [9, 4, 150]),                            # more new tokens than tokens: rows that see nothing
]


@pytest.mark.parametrize("page,hkv,group,lens,new", SHAPES)
@pytest.mark.parametrize("mod", [{}, dict(window=1), dict(window=5), dict(window=130), dict(softcap=20.0), dict(slopes=True),
                                 dict(window=64, softcap=5.0, slopes=True)])
def test_against_the_oracle(zf, page, hkv, group, lens, new, mod):
    c = Case(zf, page, hkv, group, lens, new, seed=len(lens) + hkv)
    mod = dict(mod)
    if mod.get("slopes"):
        mod["slopes"] = np.float32(2.0) ** -np.linspace(1, 8, c.hq, dtype=np.float32) * np.where(np.arange(c.hq) % 5, 1, -0.1).astype(np.float32)
    kw = {**mod, "slopes": torch.from_numpy(mod["slopes"]).cuda()} if "slopes" in mod else mod
    out, lse = zf.q4_chunk_attn(*c.args(), **kw)
    c.check(out, lse, **mod)
    assert c.cache.status_word() == 0


@pytest.mark.parametrize("scale,scales", [(0.3, (1.0, 1.0)), (-0.08, (1.0, 1.0)), (0.08, (0.37, 5.0)), (0.0, (1.0, 1.0))])
def test_scales(zf, scale, scales):
    c = Case(zf, 16, 2, 4, [260, 31], [70, 2], seed=5, scales=scales)
    out, lse = zf.q4_chunk_attn(*c.args(), scale=scale)
    c.check(out, lse, scale=scale)


def test_large_scores_keep_their_weights(zf):
    """Scores beyond 2^22, where floats lie further apart than exponents: the largest one has the weight."""
    c = Case(zf, 16, 1, 2, [300], [40], seed=9, spread=50.0)
    for scale in (3e3, 3e5, -3e5):
        out, lse = zf.q4_chunk_attn(*c.args(), scale=scale)
        q, k, v = f64(c.q), c.k[0], c.v[0]
        for t in range(40):
            for h in range(2):
                x = scale * (k[:261 + t, 0] @ q[t, h])
                order = np.argsort(x)
                gap = x[order[-1]] - x[order[-2]]
                assert np.isfinite(lse[t, h].item())
                if gap > 2.0 ** -15 * np.abs(x).max() + 40:          # one token has it all
                    want = v[order[-1], 0]
                    assert (np.abs(f64(out[t, h]) - want) <= 2.0 ** -7 * np.abs(want) + 1e-12).all()


@pytest.mark.parametrize("group,tokens", [(1, 1), (1, 16), (1, 17), (4, 4), (4, 5), (16, 1), (15, 1), (7, 2), (17, 1)])
@pytest.mark.parametrize("mod", [{}, dict(steep=1.0), dict(steep=-1.0, window=200), dict(softcap=3.0, steep=0.5), dict(window=1)])
def test_up_to_sixteen_rows_and_a_few_more(zf, group, tokens, mod):
    """Units whose rows every warp has, at every end of a context, and slopes that raise the maximum in every step."""
    lens = [tokens + n for n in (0, 1, 15, 16, 17, 111, 112, 127, 128, 129, 700)]
    c = Case(zf, 16, 2, group, lens, [tokens] * len(lens), seed=group + tokens)
    c.table[10, 40] = -1                                             # a page that is not there
    seen = [np.ones(L, bool) for L in lens]
    seen[10][640:656] = False
    mod = dict(mod)
    steep = mod.pop("steep", None)
    kw = dict(mod)
    if steep is not None:
        mod["slopes"] = np.float32(steep) * np.linspace(0.01, 1, c.hq, dtype=np.float32)
        kw["slopes"] = torch.from_numpy(mod["slopes"]).cuda()
    out, lse = zf.q4_chunk_attn(*c.args(), **kw)
    c.check(out, lse, seen=seen, **mod)
    assert c.cache.status_word() == (zf.DEV_BAD_PAGE_ID if mod.get("window", 999) > 700 - 656 else 0)       # (no window reaches it)


@pytest.mark.parametrize("window,new", [(1, 1), (40, 3), (100, 70), (129, 200)])
def test_pages_behind_the_window_may_be_gone(zf, window, new):
    c = Case(zf, 16, 2, 4, [900, 333], [new, new], seed=window)
    for b, L in enumerate(c.lens):
        c.table[b, :max(0, L - new + 1 - window) // 16] = -1
    out, lse = zf.q4_chunk_attn(*c.args(), window=window)
    c.check(out, lse, window=window)
    assert c.cache.status_word() == 0


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 200, 1000])
def test_windows_beyond_the_context(zf, window):
    """A window that reaches past the context cuts nothing, also where the first new tokens see nothing."""
    c = Case(zf, 16, 2, 4, [5, 3, 140, 300], [9, 4, 150, 20], seed=15)
    want = zf.q4_chunk_attn(*c.args())
    got = zf.q4_chunk_attn(*c.args(), window=window)
    c.check(*got)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("slopes", [False, True])
def test_units_of_all_sizes_on_one_sm(zf, slopes):
    """Many requests of few, some and many rows: each CTA goes from units of two tiles to units of one and back."""
    rng = np.random.default_rng(3)
    new = rng.choice([0, 1, 2, 4, 5, 20, 32, 33, 70], 150).tolist()
    lens = [n + int(rng.choice([0, 1, 40, 200, 600])) for n in new]
    c = Case(zf, 16, 3, 4, lens, new, seed=21)
    slope = np.float32(2.0) ** -np.linspace(1, 8, c.hq, dtype=np.float32) if slopes else None
    kw = dict(slopes=torch.from_numpy(slope).cuda()) if slopes else {}
    out, lse = zf.q4_chunk_attn(*c.args(), **kw)
    c.check(out, lse, slopes=slope)
    assert c.cache.status_word() == 0


def test_rows_of_no_request_are_left_alone(zf):
    c = Case(zf, 16, 2, 4, [50, 200], [5, 40], seed=2, lead=3, behind=6)
    out = torch.full((c.rows, c.hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.rows, c.hq), 7.0, device="cuda")
    o, l = zf.q4_chunk_attn(*c.args(), out=out, lse=lse)
    assert o.data_ptr() == out.data_ptr() and l.data_ptr() == lse.data_ptr()
    c.check(out, lse)
    for part in (slice(0, 3), slice(48, 54)):
        assert (out[part] == 7).all() and (lse[part] == 7).all()


def test_bad_pages_are_skipped(zf):
    c = Case(zf, 16, 2, 4, [200, 150], [10, 150], seed=4)
    seen = [np.ones(200, bool), np.ones(150, bool)]
    c.table[0, 3], c.table[1, 0] = 10000, -5
    seen[0][48:64], seen[1][:16] = False, False
    out, lse = zf.q4_chunk_attn(*c.args())
    c.check(out, lse, seen=seen)                                     # rows 0 .. 15 of the second see nothing
    assert c.cache.status_word() == zf.DEV_BAD_PAGE_ID


def test_bad_starts_and_lengths(zf):
    c = Case(zf, 16, 1, 4, [60, 40, 80, 30], [6, 5, 7, 4], seed=6)
    cache, q, table, lens, start = c.args()
    out, lse = torch.full((22, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((22, 4), 7.0, device="cuda")
    bad = start.clone()
    bad[4] = 23                                                      # the last request passes the rows
    zf.q4_chunk_attn(cache, q, table, lens, bad, out=out, lse=lse)
    c.check(out, lse, requests=[0, 1, 2])
    assert (out[18:] == 7).all() and cache.status_word() == zf.DEV_BAD_SEQ_LEN
    cache.status.zero_()
    bad = start.clone()
    bad[2] = 2                                                       # request 1 ends before it starts, request 2 begins there
    zf.q4_chunk_attn(cache, q, table, lens, bad)
    assert cache.status_word() == zf.DEV_BAD_SEQ_LEN
    cache.status.zero_()
    long = lens.clone()
    long[1], long[3] = -3, table.shape[1] * 16 + 1                   # clamped: nothing, and the whole row of pages
    out, lse = zf.q4_chunk_attn(cache, q, table, long, start)
    c.check(out, lse, requests=[0, 2])
    assert not out[6:11].any() and (lse[6:11] == -math.inf).all()
    assert cache.status_word() & zf.DEV_BAD_SEQ_LEN


def test_a_nan_or_infinity_stays_in_its_row(zf):
    c = Case(zf, 16, 1, 4, [300, 20], [50, 3], seed=8)
    want, wl = zf.q4_chunk_attn(*c.args())
    q = c.q.clone()
    q[7, 2, 5], q[20, 0, 100], q[51, 3, 0] = float("nan"), float("inf"), -float("inf")
    cache, _, table, lens, start = c.args()
    out, lse = zf.q4_chunk_attn(cache, q.cuda(), table, lens, start)
    hit = torch.zeros(53, 4, dtype=torch.bool)
    hit[7, 2] = hit[20, 0] = hit[51, 3] = True
    assert torch.isnan(lse.cpu()[hit]).all() and torch.isnan(out.cpu()[hit]).all()
    assert torch.equal(out.cpu()[~hit], want.cpu()[~hit]) and torch.equal(lse.cpu()[~hit], wl.cpu()[~hit])


def test_small_and_large_query_rows(zf):
    """Rows of very different size in one call: each has a power of two of its own."""
    c = Case(zf, 16, 1, 4, [200], [40], seed=11)
    f = torch.exp2(torch.randint(-60, 3, (40, 4, 1), generator=torch.Generator().manual_seed(1)).float())
    c.q = (c.q.float() * f).to(torch.bfloat16)
    c.q[3] = 0
    out, lse = zf.q4_chunk_attn(*c.args())
    c.check(out, lse)


def torch_reference(zf, cache, q, table, lens, start, page, window=0, rows=None):
    """float64 on the GPU, for contexts too long for the oracle's loops."""
    out, lse = [], []
    for b in range(len(lens)):
        L, T = lens[b], start[b + 1] - start[b]
        at = torch.arange(L, device="cuda")
        k, v = (x.view(torch.bfloat16).double() for x in
                zf.q4_read_tokens(cache, table[b][(at // page).long()].int(), (at % page).int()))
        group = q.shape[1] // k.shape[1]
        k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
        for t0 in range(0, T, 64):
            qq = q[start[b] + t0:start[b] + min(T, t0 + 64)].double()
            x = torch.einsum("thd,nhd->thn", qq, k) / math.sqrt(128)
            pos = L - T + t0 + torch.arange(qq.shape[0], device="cuda")
            hide = at[None] > pos[:, None]
            if window:
                hide |= at[None] <= pos[:, None] - window
            x.masked_fill_(hide[:, None], -math.inf)
            lse.append(torch.logsumexp(x, -1))
            out.append(torch.einsum("thn,nhd->thd", torch.softmax(x, -1), v))
    return torch.cat(out), torch.cat(lse)


@pytest.mark.parametrize("lens,new,window", [([40000], [3], 0), ([30000, 12], [200, 12], 0), ([20000, 20001], [1, 130], 5000)])
def test_units_split_over_ctas(zf, lens, new, window):
    """Long contexts and few rows: parts of units are joined."""
    page, hkv, group = 64, 2, 4
    g = torch.Generator(device="cuda").manual_seed(7)
    count = [-(-L // page) for L in lens]
    pool = sum(count)
    cache = zf.Q4Cache(pool, hkv, page)
    perm = torch.randperm(pool, generator=g, device="cuda").int()
    table = torch.full((len(lens), max(count)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(count):
        table[b, :n] = perm[at:at + n]
        at += n
    every = torch.arange(pool * page, device="cuda")
    k, v = (torch.randn(pool * page, hkv, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    zf.q4_write_tokens(cache, k, v, (every // page).int(), (every % page).int())
    start = [0] + np.cumsum(new).tolist()
    q = torch.randn(start[-1], hkv * group, 128, generator=g, device="cuda").to(torch.bfloat16)
    out, lse = zf.q4_chunk_attn(cache, q, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                torch.tensor(start, dtype=torch.int32, device="cuda"), window=window)
    want, wl = torch_reference(zf, cache, q, table, lens, start, page, window)
    # values of some 1 / sqrt(contexts): half a BF16 step and the fp16 weights' errors, which average out
    assert ((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -11 * 0.9).all()
    assert ((lse.double() - wl).abs() <= 2.0 ** -16 * 40).all()
    # the decode kernel agrees where it has the same rows
    if len(set(new)) == 1 and new[0] <= 4 and not window:
        o, l = zf.q4_decode_attn(cache, q.view(len(lens), new[0], -1, 128), table, torch.tensor(lens, dtype=torch.int32, device="cuda"))
        assert ((out.double() - o.view(out.shape).double()).abs() <= 2.0 ** -8 * o.view(out.shape).abs() + 2.0 ** -11).all()
        assert ((lse - l.view(lse.shape)).abs() <= 2.0 ** -16 * 40).all()


def test_many_requests(zf):
    """4096 requests, most without new tokens; every CTA finds its own."""
    B, page = 4096, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    new = torch.zeros(B, dtype=torch.int64)
    new[[5, 6, 900, 2047, 2048, 4095]] = torch.tensor([3, 1, 200, 40, 1, 7])
    lens = torch.full((B,), 30)
    lens[900] = 256
    table = torch.randint(0, 50, (B, 16), generator=torch.Generator().manual_seed(1), dtype=torch.int32).cuda()
    cache = zf.Q4Cache(50, 1, page)
    every = torch.arange(50 * page, device="cuda")
    k, v = (torch.randn(50 * page, 1, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    zf.q4_write_tokens(cache, k, v, (every // page).int(), (every % page).int())
    start = torch.cat((torch.zeros(1, dtype=torch.int64), new.cumsum(0)))
    q = torch.randn(int(start[-1]), 4, 128, generator=g, device="cuda").to(torch.bfloat16)
    lens[2047] = 41
    out, lse = zf.q4_chunk_attn(cache, q, table, lens.int().cuda(), start.int().cuda())
    keep = [b for b in range(B) if new[b]]
    some = [0] + new[keep].cumsum(0).tolist()
    want, wl = torch_reference(zf, cache, q, table[keep], lens[keep].tolist(), some, page)
    assert ((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -11 * 4).all()
    assert ((lse.double() - wl).abs() <= 2.0 ** -16 * 40).all()


def test_offsets_beyond_32_bits(zf):
    """Pages whose records lie beyond 4 GiB."""
    page, hkv = 128, 8
    pool = (5 << 30) // (hkv * 8 * 2304)
    cache = zf.Q4Cache(pool, hkv, page)
    g = torch.Generator(device="cuda").manual_seed(2)
    ids = torch.tensor([pool - 1, 3, pool - 2], device="cuda")
    L = 300
    at = torch.arange(L, device="cuda")
    k, v = (torch.randn(L, hkv, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    zf.q4_write_tokens(cache, k, v, ids[at // page].int(), (at % page).int())
    q = torch.randn(9, 16, 128, generator=g, device="cuda").to(torch.bfloat16)
    table = ids.int()[None]
    lens, start = torch.tensor([L], dtype=torch.int32, device="cuda"), torch.tensor([0, 9], dtype=torch.int32, device="cuda")
    out, lse = zf.q4_chunk_attn(cache, q, table, lens, start)
    want, wl = torch_reference(zf, cache, q, table, [L], [0, 9], page)
    assert ((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -11 * 4).all()
    assert ((lse.double() - wl).abs() <= 2.0 ** -16 * 40).all()


def test_same_bits_again_captured_and_on_other_streams(zf):
    c = Case(zf, 16, 2, 4, [900, 37, 129, 400], [200, 37, 1, 1], seed=12)
    args = c.args()
    need = zf.q4_chunk_workspace_size(4, c.rows, c.hq, 2, 16, c.table.shape[1])
    want = zf.q4_chunk_attn(*args)
    ws = [torch.full((need,), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]      # exactly enough, any contents
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [zf.q4_chunk_attn(*args, workspace=w, stream=s) for w, s in zip(ws * 3, streams * 3)]
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])
    with pytest.raises(zf.ZfError, match="workspace"):
        zf.q4_chunk_attn(*args, workspace=ws[0][:need - 1])
    # two graphs that share a workspace, replayed one after the other, with other lengths than captured
    cache, q, table, lens, start = args
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    graphs = []
    for kw in ({}, dict(window=50)):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            zf.q4_chunk_attn(cache, q, table, lens, start, out=out, lse=lse, workspace=ws[0], **kw)
        graphs.append(gr)
    shorter = torch.tensor([880, 37, 100, 399], dtype=torch.int32, device="cuda")
    for values in (shorter, lens.clone()):
        lens.copy_(values)
        for gr, kw in zip(graphs, ({}, dict(window=50))):
            gr.replay()
            o, l = zf.q4_chunk_attn(cache, q, table, lens, start, workspace=ws[1], **kw)
            assert torch.equal(o, out) and torch.equal(l, lse)


def test_behind_a_late_writer(zf):
    """The kernel ahead lets the next one start and then writes its lengths and rows."""
    late = H.late_writer()
    c = Case(zf, 16, 1, 4, [120, 60], [30, 2], seed=13)
    cache, q, table, lens, start = c.args()
    want = zf.q4_chunk_attn(cache, q, table, lens, start)
    d_lens, d_q = torch.zeros_like(lens), torch.zeros_like(q)
    d_start = torch.zeros_like(start)
    ws = zf.new_workspace(zf.q4_chunk_workspace_size(2, c.rows, 4, 1, 16, table.shape[1]))
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    s = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    d_lens.copy_(lens)
    assert late(start.data_ptr(), d_start.data_ptr(), 3, q.data_ptr(), d_q.data_ptr(), q.numel() // 2, 300000, s) == 0
    zf.q4_chunk_attn(cache, d_q, table, d_lens, d_start, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_more_steps_than_are_counted_are_refused(zf):
    """A page table with room for 2^30 tokens: one request of few heads is right, two of many are refused."""
    page, room = 16, 1 << 26
    for batch, hkv, ok in ((1, 1, True), (2, 32, False)):
        cache = zf.Q4Cache(4, hkv, page)
        table = torch.zeros((batch, room), dtype=torch.int32, device="cuda")
        table[:, 1] = 1
        k = torch.ones(40, hkv, 128, dtype=torch.bfloat16, device="cuda")
        at = torch.arange(20, dtype=torch.int32, device="cuda").repeat(2)
        zf.q4_write_tokens(cache, k, k, at // page, at % page)
        lens = torch.full((batch,), 20, dtype=torch.int32, device="cuda")
        start = torch.arange(batch + 1, dtype=torch.int32, device="cuda") * 3
        q = torch.ones(3 * batch, hkv, 128, dtype=torch.bfloat16, device="cuda")
        if ok:
            out, _ = zf.q4_chunk_attn(cache, q, table, lens, start)
            # (a block of ones is stored as codes of 6 and the e4m3 scale next to 1 / 6, 11 / 64: 1.03125, a BF16 value)
            assert (out == 1.03125).all()
        else:
            with pytest.raises(zf.ZfError, match="unsupported"):
                zf.q4_chunk_attn(cache, q, table, lens, start)
        assert cache.status_word() == 0


def test_a_wait_that_runs_out_reports_timeout_and_the_next_call_is_right(zf):
    """The first wait of every CTA's warps is made to run out: the call reports it and ends, and the next one, right
    behind it on the same stream, gives what it gave before."""
    c = Case(zf, 16, 2, 4, [900, 37, 129, 400], [200, 1, 4, 40], seed=14)
    args = c.args()
    want = zf.q4_chunk_attn(*args)
    for limit in (1000, 200_000):
        zf.q4_chunk_attn_wait_test(*args, wait_limit_ns=limit)
        got = zf.q4_chunk_attn(*args)
        torch.cuda.synchronize()
        assert c.cache.status_word() == zf.DEV_TIMEOUT
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        c.cache.status.zero_()
    for limit in (0, 999, 2_000_000_001):
        with pytest.raises(zf.ZfError, match="invalid argument"):
            zf.q4_chunk_attn_wait_test(*args, wait_limit_ns=limit)
    assert c.cache.status_word() == 0


@pytest.mark.parametrize("tokens,sizes", [(3, (-12, 13)), (70, (-12, 13)), (70, (-2, -1)), (70, (0, 1)), (70, (3, 4))])
@pytest.mark.parametrize("softcap", [1e-3, 0.1, 3.0, 50.0, 128.0, 128.01, 1e3, 1e4, 1e5, 1e6])
def test_caps_over_their_whole_range(zf, softcap, tokens, sizes):
    """The error of a capped score does not grow with the cap: rows of sizes from 2^-12 to 2^12, and rows alike, whose scores
    are all on one side of a cap or on both."""
    c = Case(zf, 16, 2, 4, [tokens + 200, tokens, tokens + 40], [tokens] * 3, seed=31)
    f = torch.exp2(torch.randint(*sizes, (c.rows, c.hq, 1), generator=torch.Generator().manual_seed(2)).float())
    c.q = (c.q.float() * f).to(torch.bfloat16)
    for window in (1, 0):
        out, lse = zf.q4_chunk_attn(*c.args(), softcap=softcap, window=window)
        out, lse = f64(out), lse.double().cpu().numpy()
        for b, L in enumerate(c.lens):
            a, e = c.start[b], c.start[b + 1]
            want, wl, wv, sv, mag = R.chunk_attention(f64(c.q[a:e]), c.k[b], c.v[b], L - tokens, 1 / math.sqrt(128), window, softcap)
            # a score before the cap: off by 2^-16 of its products' magnitudes (see check), which the cap does not raise;
            # after it 2^-20 of itself, or with a cap up to 128 2^-21 of that (cap - 2 cap / (1 + e), with e off by 2^-22,
            # 1 + e by 2^-24, the reciprocal by 2^-23, the result by 2^-24 of the cap); and a few roundings more in log2
            # units and back
            cap = 2.0 ** -21 * softcap if softcap <= 128 else 0.0
            off = mag * 2.0 ** -16 + 2.0 ** -20 * np.minimum(mag, softcap) + 2.0 ** -20 + cap
            tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2 * off + 2.0 ** -18)[..., None] * wv + 2.0 ** -32 * sv + 1e-30
            assert (np.abs(out[a:e] - want) <= tol).all(), (b, window, (np.abs(out[a:e] - want) / tol).max())
            tol = off + 2.0 ** -20 * (1 + np.abs(wl))                    # (window 1: lse is the score of the row's own token)
            assert (np.abs(lse[a:e] - wl) <= tol).all(), (b, window, (np.abs(lse[a:e] - wl) / tol).max())
    assert c.cache.status_word() == 0


@pytest.mark.parametrize("page,hkv,group,lens,new", SHAPES)
def test_wide_caps_against_the_oracle(zf, page, hkv, group, lens, new):
    """Caps above 128 have kernels of their own, with slopes and without."""
    c = Case(zf, page, hkv, group, lens, new, seed=len(lens) + hkv)
    slope = np.float32(2.0) ** -np.linspace(1, 8, c.hq, dtype=np.float32)
    for mod in (dict(softcap=200.0), dict(softcap=1000.0, window=64, slopes=slope)):
        kw = {**mod, "slopes": torch.from_numpy(slope).cuda()} if "slopes" in mod else mod
        out, lse = zf.q4_chunk_attn(*c.args(), **kw)
        c.check(out, lse, **mod)
    q = c.q.clone()
    q[-1, 0, 5] = float("nan")
    got = zf.q4_chunk_attn(c.cache, q.cuda(), *c.args()[2:], softcap=200.0)
    want = zf.q4_chunk_attn(*c.args(), softcap=200.0)
    hit = torch.zeros(c.rows, c.hq, dtype=torch.bool)
    hit[-1, 0] = True
    assert torch.isnan(got[0].cpu()[hit]).all() and torch.isnan(got[1].cpu()[hit]).all()
    assert torch.equal(got[0].cpu()[~hit], want[0].cpu()[~hit]) and torch.equal(got[1].cpu()[~hit], want[1].cpu()[~hit])
    assert c.cache.status_word() == 0


@pytest.mark.parametrize("batch,rows,hq,hkv", [(4096, 1, 1, 1), (16, 100000, 32, 8), (1, 3000, 28, 28)])
def test_the_limit_of_units_and_steps(zf, batch, rows, hq, hkv):
    """Refused from 7 * units * (steps + 6) = 2^31 - 1 on; below that the workspace, too small here, is looked at (nothing is
    launched)."""
    units = (rows * (hq // hkv) // 256 + batch) * hkv
    steps = -(-(2 ** 31 - 1) // (7 * units)) - 6                     # the first that is too many
    d = _desc(zf)
    d.num_kv_heads, d.page_size = hkv, 16
    call = lambda max_pages: zf.lib().zf_q4_chunk_attn(  # noqa: E731
        ctypes.byref(d), 0x10000, rows, batch, hq, 0x20000, 0x30000, max_pages, 0x40000, 0.1, 0, 0.0, None, 0x50000, 0x60000,
        0x70000, 16, None)
    assert 8 * steps * 16 < 2 ** 31 - 4096
    assert call(8 * steps - 1) == -3 and call(8 * steps) == -2
