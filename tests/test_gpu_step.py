"""Slot maps and draft verification on the GPU against the oracle, and a speculative step through all of
them: map, write, attend, verify, and the next step's map over the shortened lengths."""
import numpy as np
import pytest
import torch

from oracle import zf_step_oracle as S
from tests import helpers as H

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zf():
    return H.zf_module()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32)


def map_case(B, page, max_pages, new_max, seed, spare=True):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, max(1, max_pages * page - new_max), B)
    new = rng.integers(0, new_max + 1, B)
    held = -(-lens // page)
    if spare:
        held = np.minimum(held + rng.integers(0, 3, B), max_pages)
    pool = rng.permutation(int(held.sum()) + int((-(-(lens + new) // page)).sum()) + 3).tolist()
    table = np.full((B, max_pages), -7, np.int64)
    at = 0
    for b in range(B):
        table[b, :held[b]] = pool[at:at + held[b]]
        at += held[b]
    return table, lens, held, new, pool[at:]


def run_map(zf, table, lens, held, new, free, pos, page, max_tokens, **kw):
    t = i32(table).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    m = zf.map_tokens(t, i32(lens).cuda(), i32(held).cuda(), i32(new).cuda(), i32(free).cuda(), i32([pos]).cuda(), page,
                      max_tokens, status=status, **kw)
    return t, m, int(status)


def same_map(t, m, status, want):
    table, lens, held, pos, starts, ids, positions, seq, st = want
    assert t.cpu().tolist() == [list(map(int, r)) for r in table]
    for got, w in zip(m, (lens, held, [pos], starts, ids, positions, seq)):
        assert got.cpu().tolist() == [int(x) for x in w]
    assert status == st


@pytest.mark.parametrize("B,page,max_pages,new_max,slack", [
    (1, 16, 1, 1, 0), (1, 16, 600, 9000, 5), (7, 48, 5, 30, 1), (64, 16, 40, 5, 0), (33, 128, 9, 700, 3),
    (1024, 16, 6, 20, 2), (1025, 16, 4, 9, 7), (4096, 32, 3, 8, 0), (200, 16, 64, 1000, 11)])
def test_map_matches_the_oracle(zf, B, page, max_pages, new_max, slack):
    table, lens, held, new, free = map_case(B, page, max_pages, new_max, B + page)
    max_tokens = int(new.sum()) + slack
    want = S.map_tokens(table, lens, held, new, free, 1, page, max_tokens)
    assert want[-1] == 0
    same_map(*run_map(zf, table, lens, held, new, free, 1, page, max_tokens), want)


def test_map_in_place(zf):
    """Outputs that are the inputs themselves, across one CTA and across a cluster of 8 and 16."""
    for B, new_max, max_pages in ((5, 20, 6), (90, 400, 60), (128, 2000, 200)):
        table, lens, held, new, free = map_case(B, 16, max_pages, new_max, B)
        max_tokens = int(new.sum()) + 1
        want = S.map_tokens(table, lens, held, new, free, 0, 16, max_tokens)
        t, L, h, pos = i32(table).cuda(), i32(lens).cuda(), i32(held).cuda(), i32([0]).cuda()
        lists = [torch.empty(max_tokens, dtype=torch.int32, device="cuda") for _ in range(3)]
        out = zf.TokenMap(L, h, pos, torch.empty(B + 1, dtype=torch.int32, device="cuda"), *lists)
        m = zf.map_tokens(t, L, h, i32(new).cuda(), i32(free).cuda(), pos, 16, max_tokens, out=out)
        assert m.seq_lens.data_ptr() == L.data_ptr()
        same_map(t, m, 0, want)


def test_map_refuses_as_a_whole(zf):
    """Too few pages, too few entries, a bad free position: nothing is mapped."""
    table, lens, held, new, free = map_case(9, 16, 8, 40, 3)
    total = int(new.sum())
    need = S.map_tokens(table, lens, held, new, free, 0, 16, total)[3]
    assert need > 1
    for f, pos, most in ((free[:need - 1], 0, total), (free[:need], 1, total), (free[:need], 0, total - 1),
                         (free, -1, total), ([], 0, total)):
        want = S.map_tokens(table, lens, held, new, f, pos, 16, most)
        assert want[-1] == S.DEV_CAPACITY
        same_map(*run_map(zf, table, lens, held, new, f, pos, 16, most), want)
    big = np.full(9, 2 ** 31 - 1)                    # sums beyond 32 bits
    want = S.map_tokens(table, lens, held, big, free, 0, 16, total)
    same_map(*run_map(zf, table, lens, held, big, free, 0, 16, total), want)


def test_map_bad_requests_get_nothing(zf):
    table, lens, held, new, free = map_case(8, 16, 8, 10, 5)
    lens, held, new = lens.copy(), held.copy(), new.copy()
    lens[1], new[2], held[3], held[4], lens[5] = -4, -1, 9, -1, 8 * 16 + 1
    new[6] = 8 * 16
    lens[6] = 1
    held[6] = 1
    want = S.map_tokens(table, lens, held, new, free, 0, 16, 100)
    assert want[-1] == S.DEV_BAD_SEQ_LEN
    same_map(*run_map(zf, table, lens, held, new, free, 0, 16, 100), want)


def test_map_near_the_largest_length(zf):
    page = 48
    max_pages = (2 ** 31 - 1) // page                       # the next page's end is past 2^31
    table = torch.zeros((1, max_pages), dtype=torch.int32, device="cuda")
    L = (max_pages - 1) * page
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    m = zf.map_tokens(table, i32([L]).cuda(), i32([max_pages - 1]).cuda(), i32([40]).cuda(), i32([9, 5]).cuda(),
                      i32([1]).cuda(), page, 42, status=status)
    assert m.seq_lens.tolist() == [L + 40] and m.pages_held.tolist() == [max_pages] and m.free_pos.tolist() == [2]
    assert m.page_ids.tolist() == [5] * 40 + [-1] * 2 and m.positions.tolist() == list(range(40)) + [-1] * 2
    assert m.seq_positions.tolist() == list(range(L, L + 40)) + [-1] * 2
    assert table[0, -1].item() == 5 and table[0, :-1].abs().sum().item() == 0 and int(status) == 0


def test_map_of_nothing(zf):
    same_map(*run_map(zf, np.full((3, 2), 1), [0, 5, 32], [0, 1, 2], [0, 0, 0], [4], 0, 16, 0),
             S.map_tokens([[1, 1]] * 3, [0, 5, 32], [0, 1, 2], [0, 0, 0], [4], 0, 16, 0))
    t, m, st = run_map(zf, np.zeros((0, 2)), [], [], [], [4], 0, 16, 5)
    assert m.page_ids.tolist() == [-1] * 5 and m.token_start.tolist() == [0] and m.free_pos.tolist() == [0] and st == 0


def probs(shape, seed, sharp=2.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return torch.softmax(sharp * torch.randn(*shape, generator=g), -1).to(dtype)


def run_verify(zf, target, draft, drafts, n, uniform, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    acc, tok = zf.verify_drafts(target.cuda(), drafts.cuda(), uniform.cuda(),
                                draft_probs=None if draft is None else draft.cuda(),
                                n_drafts=None if n is None else n.cuda(), status=status, **kw)
    return acc.cpu().tolist(), tok.cpu().tolist(), int(status)


def same_verify(zf, target, draft, drafts, n, uniform):
    acc, tok, gaps, st = S.verify(target.numpy(), None if draft is None else draft.numpy(), drafts.numpy(),
                                  None if n is None else n.numpy(), uniform.numpy())
    # a drawn point within 2^-44 of a border may fall on either side: none of these inputs has one
    assert min(gaps) > 2.0 ** -44
    got = run_verify(zf, target, draft, drafts, n, uniform)
    assert got == (acc, tok, st)
    return acc, tok, st


@pytest.mark.parametrize("B,T,V,with_draft", [
    (1, 1, 1, True), (1, 4, 37, True), (3, 2, 1000, False), (5, 4, 4097, True), (2, 8, 32000, True), (1, 3, 131072, True),
    (40, 5, 5003, True), (130, 2, 2048, False), (300, 1, 515, True), (2, 64, 300, True), (1, 2, 200001, False)])
def test_verify_matches_the_oracle(zf, B, T, V, with_draft):
    rng = np.random.default_rng(V)
    target = probs((B, T + 1, V), V)
    # drafts near the target, so that runs of every length are accepted
    noise = torch.exp(0.3 * torch.randn(B, T, V, generator=torch.Generator().manual_seed(V + 1)))
    draft = target[:, :T] * noise
    draft = draft / draft.sum(-1, keepdim=True)
    source = draft if with_draft else target[:, :T]
    drafts = torch.multinomial(source.reshape(B * T, V), 1, generator=torch.Generator().manual_seed(V + 2)).view(B, T)
    drafts = drafts.to(torch.int32)
    uniform = torch.from_numpy(rng.random((B, T + 1)).astype(np.float32))
    n = i32(rng.integers(0, T + 1, B))
    for count in (None, n):
        same_verify(zf, target, draft if with_draft else None, drafts, count, uniform)


def test_verify_corners(zf):
    B, T, V = 6, 3, 700
    target, draft = probs((B, T + 1, V), 1), probs((B, T, V), 2)
    drafts = i32(np.random.default_rng(0).integers(0, V, (B, T)))
    uniform = torch.rand(B, T + 1, generator=torch.Generator().manual_seed(3))
    draft[0] = target[0, :T]                        # q = p: all accepted for u < 1
    target[1, 0] = 0                                # refused, nothing above q
    target[1, 0, 5] = 1
    draft[1, 0] = 0
    draft[1, 0, 5] = 1.5                            # p - q nowhere positive: sampled from p
    drafts[1, 0] = 9
    target[2] = 0                                   # a single token, the last
    target[2, :, V - 1] = 1
    target[3, :, :] = 0                             # mass in the first place only
    target[3, :, 0] = 1
    uniform[4] = 0
    uniform[5] = 1 - 2.0 ** -24
    same_verify(zf, target, draft, drafts, None, uniform)
    same_verify(zf, target, None, drafts, None, uniform)


def test_verify_bad_rows_and_drafts(zf):
    B, T, V = 5, 2, 300
    target, draft = probs((B, T + 1, V), 4), probs((B, T, V), 5)
    drafts = i32(np.random.default_rng(1).integers(0, V, (B, T)))
    uniform = torch.rand(B, T + 1, generator=torch.Generator().manual_seed(6))
    target[0] = 0                                   # no mass
    target[1, :, 7] = float("inf")
    target[2, :, 9] = float("nan")                  # counts as 0
    drafts[3, 0] = V
    drafts[4, 1] = -1
    n = i32([2, 2, 2, 2, 5])
    acc, tok, st = same_verify_bad(zf, target, draft, drafts, n, uniform)
    assert st == S.DEV_BAD_DRAFT | S.DEV_BAD_PROBS
    assert tok[0][acc[0]] == -1 and tok[1][acc[1]] == -1 and tok[2][acc[2]] != 9
    same_verify_bad(zf, target, None, drafts, i32([-1, 2, 2, 2, 2]), uniform)


def same_verify_bad(zf, target, draft, drafts, n, uniform):
    with np.errstate(invalid="ignore"):
        acc, tok, gaps, st = S.verify(target.numpy(), None if draft is None else draft.numpy(), drafts.numpy(), n.numpy(),
                                      uniform.numpy())
    assert min(gaps) > 2.0 ** -44
    assert run_verify(zf, target, draft, drafts, n, uniform) == (acc, tok, st)
    return acc, tok, st


def test_verify_unaligned_rows_and_lengths(zf):
    """A target whose storage starts off a 16-byte boundary, an odd vocabulary, and the shortened lengths."""
    B, T, V = 3, 2, 1001
    flat = torch.empty(B * (T + 1) * V + 1, device="cuda")
    target = probs((B, T + 1, V), 11)
    view = flat[1:].view(B, T + 1, V)
    view.copy_(target)
    draft = probs((B, T, V), 12)
    drafts = i32(np.random.default_rng(2).integers(0, V, (B, T)))
    uniform = torch.rand(B, T + 1, generator=torch.Generator().manual_seed(13))
    acc, tok, _, _ = S.verify(target.numpy(), draft.numpy(), drafts.numpy(), None, uniform.numpy())
    lens = i32([10, 20, 30]).cuda()
    a, t = zf.verify_drafts(view, drafts.cuda(), uniform.cuda(), draft_probs=draft.cuda(), seq_lens=lens, new_seq_lens=lens)
    assert a.tolist() == acc and t.tolist() == tok
    assert lens.tolist() == [L - (T - x) for L, x in zip((10, 20, 30), acc)]


def test_verify_distribution(zf):
    """Accepted or resampled, the first token is distributed as the target's: counts over 60000 draws lie
    within five standard deviations of their expectations."""
    V, N = 5, 60000
    p = torch.tensor([0.4, 0.1, 0.25, 0.05, 0.2])
    q = torch.tensor([0.1, 0.5, 0.2, 0.15, 0.05])
    g = torch.Generator().manual_seed(21)
    counts = torch.zeros(V)
    for _ in range(N // 4000):
        drafts = torch.multinomial(q, 4000, replacement=True, generator=g).view(4000, 1).to(torch.int32)
        _, tok = zf.verify_drafts(p.expand(4000, 2, V).contiguous().cuda(), drafts.cuda(), torch.rand(4000, 2, generator=g).cuda(),
                                  draft_probs=q.expand(4000, 1, V).contiguous().cuda())
        counts += torch.bincount(tok[:, 0].cpu().long(), minlength=V)
    sd = (N * p * (1 - p)).sqrt()
    assert ((counts - N * p).abs() < 5 * sd).all(), counts / N


def spec_steps(zf, c, table, lens, held, free, pos, inputs, B, T, hkv, hq, page, graph=False):
    """Two speculative steps; inputs hold each step's q, k, v, target, draft, drafts, uniform on the device."""
    new = torch.full((B,), T + 1, dtype=torch.int32, device="cuda")
    lists = [torch.empty(B * (T + 1), dtype=torch.int32, device="cuda") for _ in range(3)]
    out = zf.TokenMap(lens, held, pos, torch.empty(B + 1, dtype=torch.int32, device="cuda"), *lists)
    results = []
    for x in inputs:
        m = zf.map_tokens(table, lens, held, new, free, pos, page, B * (T + 1), out=out)
        zf.q4_write_tokens(c, x["k"], x["v"], m.page_ids, m.positions)
        o, l = zf.q4_decode_attn(c, x["q"], table, m.seq_lens)
        acc, tok = zf.verify_drafts(x["target"], x["drafts"], x["uniform"], draft_probs=x["draft"], seq_lens=lens,
                                    new_seq_lens=lens)
        results.append((o, l, acc, tok, m.page_ids.clone(), m.positions.clone()))
    return results


@pytest.mark.parametrize("graph", [False, True])
def test_a_speculative_run(zf, graph):
    """Two steps as a serving loop makes them, eager and captured, against the oracle step by step."""
    B, T, hkv, hq, page, V = 3, 3, 2, 8, 16, 400
    rng = np.random.default_rng(33)
    lens0, max_pages, pool = [30, 0, 17], 8, 30
    held0 = [-(-L // page) for L in lens0]
    perm = rng.permutation(pool).tolist()
    table0 = np.full((B, max_pages), -1)
    at = 0
    for b in range(B):
        table0[b, :held0[b]] = perm[at:at + held0[b]]
        at += held0[b]
    free = perm[at:]
    c, o = zf.Q4Cache(pool, hkv, page), S.Q4Cache(pool, hkv, page)
    old = [(int(table0[b, p // page]), p % page) for b in range(B) for p in range(lens0[b])]

    def kv(n, seed):
        g = torch.Generator().manual_seed(seed)
        return [torch.randn(n, hkv, 128, generator=g).to(torch.bfloat16).view(torch.int16) for _ in range(2)]

    k, v = kv(len(old), 1)
    zf.q4_write_tokens(c, k.cuda(), v.cuda(), [x[0] for x in old], [x[1] for x in old])
    o.write(H.np_bits(k), H.np_bits(v), [x[0] for x in old], [x[1] for x in old])
    steps = []
    for s in range(2):
        k, v = kv(B * (T + 1), 10 + s)
        g = torch.Generator().manual_seed(20 + s)
        target = probs((B, T + 1, V), 30 + s, 1.0)
        draft = target[:, :T] * torch.exp(0.5 * torch.randn(B, T, V, generator=g))
        draft = draft / draft.sum(-1, keepdim=True)
        drafts = torch.multinomial(draft.reshape(B * T, V), 1, generator=g).view(B, T).to(torch.int32)
        q = torch.randn(B, T + 1, hq, 128, generator=g).to(torch.bfloat16).view(torch.int16)
        steps.append(dict(k=k, v=v, q=q, target=target, draft=draft, drafts=drafts, uniform=torch.rand(B, T + 1, generator=g)))
    dev = [{n: x.cuda() for n, x in s.items()} for s in steps]
    state = [i32(table0).cuda(), i32(lens0).cuda(), i32(held0).cuda(), i32(free).cuda(), i32([0]).cuda()]
    args = (dev, B, T, hkv, hq, page)
    if graph:
        start = [x.clone() for x in state]
        records = c.records.clone()
        spec_steps(zf, c, *state, *args)              # warm-up
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            results = spec_steps(zf, c, *state, *args)
        for x, y in zip(state, start):
            x.copy_(y)
        c.records.copy_(records)
        gr.replay()
    else:
        results = spec_steps(zf, c, *state, *args)
    torch.cuda.synchronize()
    table, lens, held, pos = table0, lens0, held0, 0
    for x, (out, lse, acc, tok, ids, positions) in zip(steps, results):
        table, lens, held, pos, _, w_ids, w_pos, _, st = S.map_tokens(table, lens, held, [T + 1] * B, free, pos, page, B * (T + 1))
        assert st == 0 and ids.tolist() == [int(i) for i in w_ids] and positions.tolist() == w_pos
        o.write(H.np_bits(x["k"]), H.np_bits(x["v"]), w_ids, w_pos)
        ref, ref_lse, bound = S.attention(o, H.np_bits(x["q"]), np.array(table), lens, 128 ** -0.5)
        assert (np.abs(out.cpu().numpy() - ref).max(-1) <= bound * 6.0).all()
        w_acc, w_tok, gaps, _ = S.verify(x["target"].numpy(), x["draft"].numpy(), x["drafts"].numpy(), None, x["uniform"].numpy())
        assert min(gaps) > 2.0 ** -44
        assert acc.tolist() == w_acc and tok.tolist() == w_tok
        lens = [L - (T - a) for L, a in zip(lens, w_acc)]
    assert (c.records.cpu().numpy() == o.records).all()
    assert state[1].tolist() == lens and state[2].tolist() == held and state[4].tolist() == [pos]
    assert c.status_word() == 0
