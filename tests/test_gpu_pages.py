"""Forking, releasing and compacting pages against the oracle, whole numbers exactly; copies byte by byte; and a serving
loop that uses them with the other calls."""
import numpy as np
import pytest
import torch

from oracle import zf_serve_oracle as R
from tests import helpers as H

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zf():
    return H.zf_module()


def dev(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


class Pool:
    """Requests over a shuffled pool, some rows empty."""

    def __init__(self, B, max_pages, page, seed, empty=0.4, spare=0.2, most=None):
        rng = np.random.default_rng(seed)
        self.page, self.B = page, B
        self.held = (rng.integers(0, (most or max_pages) + 1, B) * (rng.random(B) >= empty)).tolist()
        self.lens = [int(rng.integers(max(0, h - 1) * page * (rng.random() > spare), h * page + 1)) if h else 0 for h in self.held]
        used = sum(self.held)
        self.pool = used + int(rng.integers(1, 2 * B + 2))
        perm = rng.permutation(self.pool)
        self.table, at = rng.integers(-5, self.pool + 5, (B, max_pages)).astype(np.int32), 0     # junk past the pages held
        for b, h in enumerate(self.held):
            self.table[b, :h] = perm[at:at + h]
            at += h
        # a list over the whole pool: what is held lies before pos
        self.free, self.pos = np.concatenate((np.full(used, -7), perm[at:])).tolist(), used
        self.rng = rng


def run_fork(zf, p, src, dst, alias=False):
    want = R.fork(p.table, p.lens, p.held, src, dst, p.free, p.pos, p.page)
    table, lens, held, pos, status = dev(p.table), dev(p.lens), dev(p.held), dev([p.pos]), word()
    out = None
    if alias:
        out = zf.Fork(lens, held, pos, torch.empty(len(src), dtype=torch.int32, device="cuda"),
                      torch.empty(len(src), dtype=torch.int32, device="cuda"))
    f = zf.fork_requests(table, lens, held, dev(src), dev(dst), dev(p.free), pos, p.page, out=out, status=status)
    assert (table.cpu().numpy() == want[0]).all()
    for got, w in zip((f.seq_lens, f.pages_held), want[1:3]):
        assert got.tolist() == w
    assert f.free_pos.tolist() == [want[3]] and f.copy_src.tolist() == want[4] and f.copy_dst.tolist() == want[5]
    assert int(status.item()) == want[6]
    return want


@pytest.mark.parametrize("B,max_pages,page,n", [(2, 1, 16, 1), (7, 3, 48, 3), (64, 70, 16, 30), (300, 600, 64, 200), (4096, 5, 16, 4096)])
@pytest.mark.parametrize("alias", [False, True])
def test_fork(zf, B, max_pages, page, n, alias):
    p = Pool(B, max_pages, page, B)
    rows = [b for b in range(B) if p.held[b] == 0 and p.lens[b] == 0]
    full = [b for b in range(B) if p.held[b]] or [0]
    dst = p.rng.permutation(rows)[:n].tolist()
    src = p.rng.choice(full, len(dst)).tolist()
    run_fork(zf, p, src, dst, alias)


def test_fork_refusals(zf):
    p = Pool(40, 6, 16, 3)
    p.held[0], p.lens[0], p.held[1], p.lens[1] = 0, 0, 2, 20
    p.held[2], p.lens[2], p.held[3], p.lens[3] = 1, 17, 7, 3          # too few pages for the length; more than the row has
    p.held[4], p.lens[4], p.held[5], p.lens[5] = 3, -1, 0, 0
    p.held[6], p.lens[6] = 0, 0
    src = [1, 1, 1, 2, 3, 4, -1, 40, 1, 1, 5, 0, 1]
    dst = [0, 0, 1, 5, 5, 5, 5, 5, 40, -1, 6, 1, 6]
    run_fork(zf, p, src, dst)
    p = Pool(40, 6, 16, 4)
    rows = [b for b in range(40) if p.held[b] == 0]
    src = [next(b for b in range(40) if p.lens[b] % 16)] * len(rows)
    p.pos = len(p.free) - len(rows)
    assert run_fork(zf, p, src, rows)[6] == 0                         # exactly enough
    p.pos += 1
    assert run_fork(zf, p, src, rows)[6] == R.DEV_CAPACITY            # one too few: nothing is forked
    p.pos = -1
    run_fork(zf, p, src, rows)
    run_fork(zf, p, [], [])


def run_release(zf, p, gone, alias=False):
    want = R.release(p.table, p.lens, p.held, gone, p.free, p.pos, p.pool)
    table, lens, held, pos, free, status = dev(p.table), dev(p.lens), dev(p.held), dev([p.pos]), dev(p.free), word()
    ws = torch.full((zf.release_workspace_size(p.pool),), 200, dtype=torch.uint8, device="cuda")
    r = zf.release_requests(table, lens, held, dev(gone), free, pos, p.pool, out=zf.Release(lens, held, pos) if alias else None,
                            status=status, workspace=ws)
    assert (r.seq_lens.tolist(), r.pages_held.tolist(), free.tolist(), r.free_pos.tolist()[0], int(status.item())) == want
    assert (table.cpu().numpy() == p.table).all()
    return want


def share(p):
    """Rows in pairs begin with the same pages."""
    for b in range(1, p.B, 2):
        k = min(p.held[b], p.held[b - 1]) // 2 + (b % 3 == 0)
        k = min(k, p.held[b], p.held[b - 1])
        p.table[b, :k] = p.table[b - 1, :k]


@pytest.mark.parametrize("B,max_pages", [(1, 1), (5, 4), (64, 70), (300, 600), (4096, 5)])
@pytest.mark.parametrize("alias", [False, True])
def test_release(zf, B, max_pages, alias):
    p = Pool(B, max_pages, 16, B + 1, empty=0.1)
    share(p)
    for part in (0.0, 0.3, 1.0):
        gone = (p.rng.random(B) < part).astype(int) * p.rng.integers(1, 9, B)
        run_release(zf, p, gone.tolist(), alias)


def test_release_refusals(zf):
    p = Pool(20, 6, 16, 5, empty=0)
    share(p)
    p.table[3, 0], p.table[4, 0] = p.pool, -1                         # no pages of the pool
    p.held[5], p.held[6] = -2, 9
    run_release(zf, p, [1] * 20)
    run_release(zf, p, [0] * 20)
    p = Pool(20, 6, 16, 6, empty=0)
    need = len(R.release(p.table, p.lens, p.held, [1] * 20, p.free, p.pos, p.pool)[2])
    p.pos = sum(p.held) - 1
    assert run_release(zf, p, [1] * 20)[4] == R.DEV_CAPACITY and need
    p.pos = len(p.free) + 1
    assert run_release(zf, p, [1] * 20)[4] == R.DEV_CAPACITY


def run_compact(zf, p, alias=False):
    want = R.compact(p.table, p.held, p.pool)
    table, status = dev(p.table), word()
    ws = torch.full((zf.compact_workspace_size(p.pool),), 200, dtype=torch.uint8, device="cuda")
    out = None
    if alias:
        e = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
        out = zf.Compaction(table, e(p.pool), e(1), e(p.pool // 2), e(p.pool // 2))
    c = zf.compact_pages(table, dev(p.held), p.pool, out=out, status=status, workspace=ws)
    assert (c.page_table.cpu().numpy() == want[0]).all()
    assert c.free_pages.tolist() == want[1] and c.free_pos.tolist() == [want[2]]
    assert c.copy_src.tolist() == want[3] and c.copy_dst.tolist() == want[4] and int(status.item()) == want[5]


@pytest.mark.parametrize("B,max_pages", [(1, 1), (5, 4), (64, 70), (300, 600), (4096, 5)])
@pytest.mark.parametrize("alias", [False, True])
def test_compact(zf, B, max_pages, alias):
    p = Pool(B, max_pages, 16, B + 2, empty=0.3, most=max(1, max_pages // 2))
    share(p)
    run_compact(zf, p, alias)
    p.held = [h * (b % 4 == 0) for b, h in enumerate(p.held)]          # most of the pool is unused
    run_compact(zf, p, alias)
    p.held = [0] * B
    run_compact(zf, p, alias)


def test_compact_refusals_and_a_full_pool(zf):
    p = Pool(20, 6, 16, 7, empty=0)
    p.table[3, 0], p.table[4, 0] = p.pool, -1
    p.held[5], p.held[6] = -2, 9
    run_compact(zf, p)
    p = Pool(20, 6, 16, 8, empty=0)
    p.pool = sum(p.held)
    p.table[:] = p.table % p.pool
    run_compact(zf, p)
    for pool in (0, 1, 2):
        p.pool = pool
        run_compact(zf, p)


@pytest.mark.parametrize("page,hkv", [(16, 1), (48, 3), (128, 8)])
def test_copy(zf, page, hkv):
    g = torch.Generator().manual_seed(1)
    pool = 60
    cache = zf.Q4Cache(pool, hkv, page, records=torch.randint(0, 255, (pool, hkv, page // 16, 2304), dtype=torch.uint8, generator=g).cuda())
    before = cache.records.clone()
    perm = torch.randperm(pool, generator=g).int()
    src, dst = perm[:25].clone(), perm[25:50].clone()
    src[3:6], dst[3:6] = -1, -1
    src[7] = src[8]                                                   # one source twice
    zf.q4_copy_pages(cache, src.cuda(), dst.cuda())
    want = before.clone()
    live = src >= 0
    want[dst[live].long()] = before[src[live].long()]
    assert torch.equal(cache.records, want) and cache.status_word() == 0
    zf.q4_copy_pages(cache, src[:0].cuda(), dst[:0].cuda())
    zf.q4_copy_pages(cache, dev([-1, 60, 2, -2, 3]), dev([4, 5, 60, -2, 3]))
    assert torch.equal(cache.records, want) and cache.status_word() == zf.DEV_BAD_PAGE_ID


def test_copy_of_long_lists_and_beyond_4_gib(zf):
    page, hkv = 128, 8
    pool = (5 << 30) // (hkv * 8 * 2304)
    cache = zf.Q4Cache(pool, hkv, page)
    cache.records[3] = 17
    cache.records[pool - 1] = 23
    src, dst = torch.full((200000,), -1, dtype=torch.int32), torch.full((200000,), -1, dtype=torch.int32)
    src[5], dst[5], src[199999], dst[199999] = 3, pool - 2, pool - 1, 0
    zf.q4_copy_pages(cache, src.cuda(), dst.cuda())
    assert (cache.records[pool - 2] == 17).all() and (cache.records[0] == 23).all()
    assert int(cache.records[1:3].sum()) == 0 and int(cache.records[pool - 3].sum()) == 0


@pytest.mark.parametrize("graph", [False, True])
def test_a_serving_loop(zf, graph):
    """Prompts in chunks, forked answers, a speculative step from sampled distributions, requests released, pages moved
    together: every request's attention equals that over a cache of its own, bit by bit, and no page is lost."""
    B, HKV, HQ, PAGE, V, MAXP = 6, 2, 8, 16, 500, 12
    pool = B * MAXP
    gen = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    cache, status = zf.Q4Cache(pool, HKV, PAGE), word()
    table = torch.full((B, MAXP), -1, dtype=torch.int32, device="cuda")
    lens, held, pos = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (B, B, 1))
    free = torch.randperm(pool, generator=gen, device="cuda").int()
    history = [[] for _ in range(B)]                                   # (k, v) of every token of a request

    def place(new):
        new_t = dev(new)
        n = sum(new)
        m = zf.map_tokens(table, lens, held, new_t, free, pos, PAGE, n, status=status)
        for t, s in ((lens, m.seq_lens), (held, m.pages_held), (pos, m.free_pos)):
            t.copy_(s)
        k, v, q = rand(n, HKV, 128), rand(n, HKV, 128), rand(n, HQ, 128)
        zf.q4_write_tokens(cache, k, v, m.page_ids, m.positions)
        out, lse = torch.empty(n, HQ, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(n, HQ, device="cuda")
        if graph:
            g = torch.cuda.CUDAGraph()
            ws = zf.new_workspace(zf.q4_chunk_workspace_size(B, n, HQ, HKV, PAGE, MAXP))
            with torch.cuda.graph(g):
                zf.q4_chunk_attn(cache, q, table, lens, m.token_start, out=out, lse=lse, workspace=ws)
            g.replay()
        else:
            zf.q4_chunk_attn(cache, q, table, lens, m.token_start, out=out, lse=lse)
        at = 0
        for b, c in enumerate(new):
            history[b] += [(k[i], v[i]) for i in range(at, at + c)]
            at += c
        alone(q, new, out, lse)
        return m

    def alone(q, new, out, lse):
        at = 0
        for b, c in enumerate(new):
            L = len(history[b])
            assert int(lens[b]) == L
            if c:
                own = zf.Q4Cache(-(-L // PAGE), HKV, PAGE)
                ids = torch.arange(L, device="cuda")
                zf.q4_write_tokens(own, torch.stack([x[0] for x in history[b]]), torch.stack([x[1] for x in history[b]]),
                                   (ids // PAGE).int(), (ids % PAGE).int())
                rows = torch.arange(own.num_pages, device="cuda").int()[None]
                o, l = zf.q4_chunk_attn(own, q[at:at + c], rows, dev([L]), dev([0, c]))
                assert torch.allclose(out[at:at + c].float(), o.float(), rtol=2.0 ** -7, atol=2.0 ** -10)
                assert torch.allclose(lse[at:at + c], l, atol=2.0 ** -14)
            at += c

    def consistent():
        pages = {int(p) for b in range(B) for p in table[b, :int(held[b])]}
        rest = free[int(pos):].tolist()
        assert len(set(rest)) == len(rest) and not pages & set(rest) and len(pages) + len(rest) == pool
        assert int(status.item()) == 0 and cache.status_word() == 0

    place([40, 0, 25, 0, 0, 0])
    place([13, 0, 0, 0, 0, 0])                                         # the first prompt's second chunk: 53 tokens
    consistent()
    f = zf.fork_requests(table, lens, held, dev([0, 0, 2]), dev([1, 4, 5]), free, pos, PAGE, status=status)
    zf.q4_copy_pages(cache, f.copy_src, f.copy_dst)
    for t, s in ((lens, f.seq_lens), (held, f.pages_held), (pos, f.free_pos)):
        t.copy_(s)
    for d, s in ((1, 0), (4, 0), (5, 2)):
        history[d] = list(history[s])
    assert table[1, :3].tolist() == table[0, :3].tolist() and int(table[1, 3]) != int(table[0, 3])
    consistent()
    # a speculative step: two drafts each, target and draft distributions from logits
    m = place([3, 3, 3, 0, 3, 3])
    logits, guess = rand(B * 3, V).float() * 3, rand(B * 2, V).float() * 3
    target, proposal = torch.empty(B * 3, V, device="cuda"), torch.empty(B * 2, V, device="cuda")
    p90 = torch.full((B * 3,), 0.9, device="cuda")
    assert zf.sample_tokens(logits, top_p=p90, probs=target, status=status) is None
    u = torch.rand(B * 2, generator=gen, device="cuda")
    drafts = zf.sample_tokens(guess, u, top_p=p90[:B * 2], probs=proposal, status=status)
    acc, tok = zf.verify_drafts(target.view(B, 3, V), drafts.view(B, 2), torch.rand(B, 3, generator=gen, device="cuda"),
                                draft_probs=proposal.view(B, 2, V), seq_lens=m.seq_lens, new_seq_lens=lens,
                                status=status, token_start=m.token_start)
    for b in range(B):
        if b != 3:
            drop = 2 - int(acc[b])
            history[b] = history[b][:len(history[b]) - drop]
            assert 0 <= int(tok[b, int(acc[b])]) < V and float(target.view(B, 3, V)[b, int(acc[b]), int(tok[b, int(acc[b])])]) > 0
    place([1, 1, 0, 0, 1, 1])
    consistent()
    r = zf.release_requests(table, lens, held, dev([1, 0, 0, 0, 0, 1]), free, pos, pool, status=status)
    for t, s in ((lens, r.seq_lens), (held, r.pages_held), (pos, r.free_pos)):
        t.copy_(s)
    history[0], history[5] = [], []
    consistent()
    place([20, 2, 17, 5, 1, 0])                                        # the first row is another request's now
    c = zf.compact_pages(table, held, pool, status=status)
    zf.q4_copy_pages(cache, c.copy_src, c.copy_dst)
    used = int(c.free_pos)
    assert used == len({int(p) for b in range(B) for p in table[b, :int(held[b])]})
    table.copy_(c.page_table)
    free.copy_(c.free_pages)
    pos.copy_(c.free_pos)
    assert max(int(p) for b in range(B) for p in table[b, :int(held[b])]) == used - 1
    consistent()
    place([1, 1, 33, 2, 1, 7])
    consistent()


def test_behind_a_late_writer(zf):
    """The kernel ahead lets the next one start and then writes what that one reads."""
    late = H.late_writer()
    p = Pool(40, 50, 16, 31, empty=0.3)
    share(p)
    s = torch.cuda.current_stream().cuda_stream
    table, lens, held = dev(p.table), dev(p.lens), dev(p.held)
    src = [b for b in range(40) if p.held[b]][:6]
    dst = [b for b in range(40) if not p.held[b]][:6]
    n = min(len(src), len(dst))
    src, dst = src[:n], dst[:n]
    free, pos = dev(p.free), dev([p.pos])
    gone = dev([b % 2 for b in range(40)])

    def behind(small, big, call):
        d_small, d_big = torch.zeros_like(small), torch.zeros_like(big)
        torch.cuda.synchronize()
        assert late(small.data_ptr(), d_small.data_ptr(), small.numel(), big.data_ptr(), d_big.data_ptr(), big.numel(), 300000, s) == 0
        out = call(d_small, d_big)
        torch.cuda.synchronize()
        return out

    want = R.fork(p.table, p.lens, p.held, src, dst, p.free, p.pos, 16)
    f = behind(dev(src), table, lambda a, t: (zf.fork_requests(t, lens, held, a, dev(dst), free, pos, 16), t))
    assert (f[1].cpu().numpy() == want[0]).all() and f[0].copy_src.tolist() == want[4] and f[0].seq_lens.tolist() == want[1]
    wl, wh, wf, wp, _ = R.release(p.table, p.lens, p.held, gone.tolist(), p.free, p.pos, p.pool)
    ws = torch.empty(zf.release_workspace_size(p.pool), dtype=torch.uint8, device="cuda")
    r = behind(gone, table, lambda a, t: zf.release_requests(t, lens, held, a, free, pos, p.pool, workspace=ws))
    assert r.seq_lens.tolist() == wl and free.tolist() == wf and r.free_pos.tolist() == [wp]
    want = R.compact(p.table, p.held, p.pool)
    wc = torch.empty(zf.compact_workspace_size(p.pool), dtype=torch.uint8, device="cuda")
    c = behind(held, table, lambda h, t: zf.compact_pages(t, h, p.pool, workspace=wc))
    assert (c.page_table.cpu().numpy() == want[0]).all() and c.copy_src.tolist() == want[3]
    cache = zf.Q4Cache(8, 1, 16)
    cache.records.copy_(torch.randint(0, 255, cache.records.shape, dtype=torch.uint8, device="cuda"))
    before = cache.records.clone().view(8, -1)
    behind(dev([5, 2]), dev([0, 7]), lambda a, b: zf.q4_copy_pages(cache, a, b))
    after = cache.records.view(8, -1)
    assert torch.equal(after[0], before[5]) and torch.equal(after[7], before[2]) and torch.equal(after[1:7], before[1:7])


def test_two_streams_at_once(zf):
    """The same calls on two streams, each with its own workspace and outputs."""
    p = Pool(200, 300, 16, 33, empty=0.2)
    share(p)
    table, lens, held, gone = dev(p.table), dev(p.lens), dev(p.held), dev([b % 3 == 0 for b in range(200)])
    want = R.release(p.table, p.lens, p.held, gone.tolist(), p.free, p.pos, p.pool)
    packed = R.compact(p.table, p.held, p.pool)
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [torch.empty(zf.release_workspace_size(p.pool), dtype=torch.uint8, device="cuda") for _ in range(2)]
    wc = [torch.empty(zf.compact_workspace_size(p.pool), dtype=torch.uint8, device="cuda") for _ in range(2)]
    lists = [[dev(p.free) for _ in range(4)] for _ in range(2)]
    pos = dev([p.pos])
    torch.cuda.synchronize()
    done = [[], []]
    for k in range(4):
        for i, s in enumerate(streams):
            done[i].append((zf.release_requests(table, lens, held, gone, lists[i][k], pos, p.pool, workspace=ws[i], stream=s),
                            zf.compact_pages(table, held, p.pool, workspace=wc[i], stream=s)))
    torch.cuda.synchronize()
    for i in range(2):
        for k in range(4):
            r, c = done[i][k]
            assert r.pages_held.tolist() == want[1] and lists[i][k].tolist() == want[2] and r.free_pos.tolist() == [want[3]]
            assert (c.page_table.cpu().numpy() == packed[0]).all() and c.free_pages.tolist() == packed[1]
