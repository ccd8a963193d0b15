"""The calls of a speculative step in a row (map, write, attend, verify) when requests get no places, and when they
have different numbers of drafts, over several steps, eager and captured, against the oracle step by step."""
import numpy as np
import pytest
import torch

from oracle import zf_step_oracle as S
from tests import helpers as H

pytestmark = pytest.mark.gpu

HKV, HQ, PAGE, V = 2, 8, 16, 300


@pytest.fixture(scope="module")
def zf():
    return H.zf_module()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32)


class Loop:
    """A serving loop's state on the GPU and in the oracle, and one step of each."""

    def __init__(self, zf, B, T, lens, max_pages, pool, seed, graph):
        self.zf, self.B, self.T, self.graph = zf, B, T, graph
        perm = np.random.default_rng(seed).permutation(pool).tolist()
        held = [-(-L // PAGE) for L in lens]
        table, at = np.full((B, max_pages), -1), 0
        for b in range(B):
            table[b, :held[b]] = perm[at:at + held[b]]
            at += held[b]
        self.table, self.lens, self.held, self.free, self.pos = table, list(lens), held, perm[at:], 0
        self.c, self.o = zf.Q4Cache(pool, HKV, PAGE), S.Q4Cache(pool, HKV, PAGE)
        old = [(int(table[b, p // PAGE]), p % PAGE) for b in range(B) for p in range(lens[b])]
        g = torch.Generator().manual_seed(seed)
        k, v = (torch.randn(len(old), HKV, 128, generator=g).to(torch.bfloat16).view(torch.int16) for _ in range(2))
        zf.q4_write_tokens(self.c, k.cuda(), v.cuda(), [x[0] for x in old], [x[1] for x in old])
        self.o.write(H.np_bits(k), H.np_bits(v), [x[0] for x in old], [x[1] for x in old])
        self.d_table, self.d_lens, self.d_held = i32(table).cuda(), i32(lens).cuda(), i32(held).cuda()
        self.d_free, self.d_pos = i32(self.free).cuda(), i32([0]).cuda()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        n = B * (T + 1)
        lists = [torch.empty(n, dtype=torch.int32, device="cuda") for _ in range(3)]
        self.out = zf.TokenMap(self.d_lens, self.d_held, self.d_pos, torch.empty(B + 1, dtype=torch.int32, device="cuda"), *lists)
        self.x, self.captured = None, None

    def call(self):
        """The four calls, on the tensors of self.x."""
        zf, x = self.zf, self.x
        m = zf.map_tokens(self.d_table, self.d_lens, self.d_held, x["new"], self.d_free, self.d_pos, PAGE,
                          self.B * (self.T + 1), out=self.out, status=self.status)
        zf.q4_write_tokens(self.c, x["k"], x["v"], m.page_ids, m.positions)
        out, lse = zf.q4_decode_attn(self.c, x["q"], self.d_table, m.seq_lens)
        acc, tok = zf.verify_drafts(x["target"], x["drafts"], x["uniform"], draft_probs=x["draft"], n_drafts=x.get("n"),
                                    seq_lens=m.seq_lens, new_seq_lens=m.seq_lens, token_start=m.token_start,
                                    status=self.status)
        return out, lse, acc, tok

    def step(self, x):
        """One step on both sides; the oracle's status."""
        B, T = self.B, self.T
        dev = {n: t.cuda() for n, t in x.items()}
        self.status.zero_()
        if not self.graph:
            self.x = dev
            out, lse, acc, tok = self.call()
        else:
            if self.captured is None:
                self.x = dev
                keep = [t.clone() for t in (self.d_table, self.d_lens, self.d_held, self.d_pos, self.c.records)]
                self.call()                                              # warm-up
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    res = self.call()
                self.captured = g, res
                for t, was in zip((self.d_table, self.d_lens, self.d_held, self.d_pos, self.c.records), keep):
                    t.copy_(was)
                self.status.zero_()
            for n, t in dev.items():
                self.x[n].copy_(t)
            self.captured[0].replay()
            out, lse, acc, tok = self.captured[1]
        torch.cuda.synchronize()
        table, lens, held, pos, starts, ids, positions, _, st = S.map_tokens(
            self.table, self.lens, self.held, x["new"].tolist(), self.free, self.pos, PAGE, B * (T + 1))
        self.o.write(H.np_bits(x["k"]), H.np_bits(x["v"]), ids, positions)
        got = np.diff(starts) > 0
        ref, ref_lse, bound = S.attention(self.o, H.np_bits(x["q"]), np.array(table), lens, 128 ** -0.5)
        off = np.abs(out.cpu().numpy() - ref).max(-1)
        assert (off <= bound * 6.0)[got].all()
        w_acc, w_tok, w_lens, gaps, vst = S.verify_step(
            x["target"].numpy(), x["draft"].numpy(), x["drafts"].numpy(), x["n"].numpy() if "n" in x else None,
            x["uniform"].numpy(), starts, lens)
        assert min(gaps) > 2.0 ** -44
        assert acc.tolist() == w_acc and tok.tolist() == w_tok
        self.table, self.lens, self.held, self.pos = np.array(table), w_lens, held, pos
        assert self.d_table.cpu().tolist() == self.table.tolist() and self.d_held.tolist() == held
        assert self.d_lens.tolist() == w_lens and self.d_pos.tolist() == [pos]
        assert (self.c.records.cpu().numpy() == self.o.records).all()
        assert int(self.status) == st | vst and self.c.status_word() == 0
        self.accepted = w_acc
        return st | vst

    def step_accepted(self, x):
        assert self.step(x) == 0
        return self.accepted


def inputs(B, T, seed, new=None):
    g = torch.Generator().manual_seed(seed)
    k, v = (torch.randn(B * (T + 1), HKV, 128, generator=g).to(torch.bfloat16).view(torch.int16) for _ in range(2))
    q = torch.randn(B, T + 1, HQ, 128, generator=g).to(torch.bfloat16).view(torch.int16)
    target = torch.softmax(torch.randn(B, T + 1, V, generator=g), -1)
    draft = target[:, :T] * torch.exp(0.5 * torch.randn(B, T, V, generator=g))
    draft = draft / draft.sum(-1, keepdim=True)
    drafts = torch.multinomial(draft.reshape(B * T, V), 1, generator=g).view(B, T).to(torch.int32)
    return dict(k=k, v=v, q=q, target=target, draft=draft, drafts=drafts, uniform=torch.rand(B, T + 1, generator=g),
                new=i32([T + 1] * B if new is None else new))


@pytest.mark.parametrize("graph", [False, True])
def test_steps_without_pages_lose_nothing(zf, graph):
    """Every request's next token needs a page and none is free: two steps are refused as a whole and leave lengths
    and cache as they were; once pages are free the same loop goes on."""
    B, T = 3, 3
    loop = Loop(zf, B, T, [32, 16, 48], 8, 12, 51, graph)
    loop.pos = len(loop.free)
    loop.d_pos.fill_(loop.pos)
    for s in range(2):
        assert loop.step(inputs(B, T, 60 + s)) == S.DEV_CAPACITY
        assert loop.lens == [32, 16, 48]
    loop.pos = 0
    loop.d_pos.zero_()
    for s in range(3):
        assert loop.step(inputs(B, T, 70 + s)) == 0
    assert all(L >= first + 3 for L, first in zip(loop.lens, [32, 16, 48]))


@pytest.mark.parametrize("graph", [False, True])
def test_refused_and_idle_requests_lose_nothing(zf, graph):
    """One request whose table is full is refused step after step, one has no new tokens; the others go on."""
    B, T = 4, 3
    loop = Loop(zf, B, T, [32, 128, 16, 5], 8, 20, 52, graph)
    for s in range(3):
        assert loop.step(inputs(B, T, 80 + s, [T + 1, T + 1, T + 1, 0])) == S.DEV_BAD_SEQ_LEN
        assert loop.lens[1] == 128 and loop.lens[3] == 5
    assert loop.lens[0] >= 35 and loop.lens[2] >= 19


@pytest.mark.parametrize("vocab", [40, 5001, 32000])
def test_places_that_are_no_steps(zf, vocab):
    """Counts of places from a negative one to a prompt's, for one CTA and for clusters; lengths shorter than what
    is taken off them become 0, with and without places."""
    T, lens = 3, [50, 50, 50, 50, 2, 0]
    places = [4, 0, 5, -2, 4, 4]
    B = len(lens)
    g = torch.Generator().manual_seed(vocab)
    target = torch.softmax(torch.randn(B, T + 1, vocab, generator=g), -1)
    drafts = torch.randint(0, vocab, (B, T), generator=g).to(torch.int32)
    uniform = torch.rand(B, T + 1, generator=g)
    starts = np.concatenate(([0], np.cumsum(places)))
    want = S.verify_step(target.numpy(), None, drafts.numpy(), None, uniform.numpy(), starts, lens)
    assert want[0][1:4] == [0] * 3 and want[2][1:4] == [50] * 3 and min(want[3]) > 2.0 ** -44
    assert want[4] == S.DEV_BAD_DRAFT | S.DEV_BAD_SEQ_LEN
    for first, out in ((i32(lens).cuda(), torch.empty(B, dtype=torch.int32, device="cuda")), (i32(lens).cuda(), None)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = first if out is None else out
        acc, tok = zf.verify_drafts(target.cuda(), drafts.cuda(), uniform.cuda(), seq_lens=first, new_seq_lens=out,
                                    token_start=i32(starts).cuda(), status=status)
        assert acc.tolist() == want[0] and tok.tolist() == want[1] and out.tolist() == want[2] and int(status) == want[4]
    acc, tok, _, _ = S.verify(target.numpy(), None, drafts.numpy(), None, uniform.numpy())
    after = [L - (T - a) for L, a in zip(lens, acc)]
    assert min(after) < 0
    status, out = torch.zeros(1, dtype=torch.int32, device="cuda"), i32(lens).cuda()
    a, t = zf.verify_drafts(target.cuda(), drafts.cuda(), uniform.cuda(), seq_lens=out, new_seq_lens=out, status=status)
    assert a.tolist() == acc and t.tolist() == tok
    assert out.tolist() == [max(L, 0) for L in after] and int(status) == S.DEV_BAD_SEQ_LEN


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("padded", [True, False])
def test_ragged_drafts_leave_no_padding(zf, padded, graph):
    """0 to T drafts per request, with T + 1 places for every request or one more than its drafts: after every step a
    request holds its last token and the accepted drafts and nothing else."""
    B, T = 5, 4
    loop = Loop(zf, B, T, [20, 0, 33, 15, 64], 8, 40, 53, graph)
    rng = np.random.default_rng(54)
    for s in range(5):
        n = [0, 0, 0, 0, 0] if s == 2 else rng.permutation([0, 1, 2, T, T]).tolist()
        x = inputs(B, T, 90 + s, [T + 1] * B if padded else [k + 1 for k in n])
        x["n"] = i32(n)
        before, kept = list(loop.lens), loop.step_accepted(x)
        assert loop.lens == [L + 1 + a for L, a in zip(before, kept)] and all(a <= k for a, k in zip(kept, n))


def test_drafts_without_places(zf):
    """More drafts than places: only the placed ones count, and the status word says so; without n_drafts the places
    decide."""
    T, lens, places, n = 4, [50, 50, 50, 50], [2, 1, 5, 3], [3, 0, 5, -1]
    B, vocab = len(lens), 100
    g = torch.Generator().manual_seed(1)
    target = torch.softmax(torch.randn(B, T + 1, vocab, generator=g), -1)
    drafts = target[:, :T].argmax(-1).to(torch.int32)
    uniform = torch.full((B, T + 1), 2.0 ** -10)               # every draft is accepted
    starts = np.concatenate(([0], np.cumsum(places)))
    for count in (n, None):
        want = S.verify_step(target.numpy(), None, drafts.numpy(), count, uniform.numpy(), starts, lens)
        assert want[0] == ([1, 0, 4, 0] if count else [1, 0, 4, 2]) and want[2] == ([50, 50, 50, 48] if count else [50] * 4)
        status, out = torch.zeros(1, dtype=torch.int32, device="cuda"), i32(lens).cuda()
        acc, tok = zf.verify_drafts(target.cuda(), drafts.cuda(), uniform.cuda(), n_drafts=None if count is None else i32(n).cuda(),
                                    seq_lens=out, new_seq_lens=out, token_start=i32(starts).cuda(), status=status)
        assert acc.tolist() == want[0] and tok.tolist() == want[1] and out.tolist() == want[2]
        assert int(status) == want[4] == (S.DEV_BAD_DRAFT if count else 0)


def test_two_loops_at_once_on_streams_of_their_own(zf):
    """Two loops whose steps overlap on two streams: every call of a step is ordered on its loop's stream."""
    B, T = 3, 3
    loops = [Loop(zf, B, T, lens, 8, 20, 55 + i, False) for i, lens in enumerate(([30, 5, 17], [16, 0, 40]))]
    streams = [torch.cuda.Stream() for _ in loops]
    steps = [[inputs(B, T, 200 + 10 * i + s) for s in range(2)] for i in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for s in range(2):
        for i, (loop, stream) in enumerate(zip(loops, streams)):
            with torch.cuda.stream(stream):
                torch.cuda._sleep(2_000_000)                 # the streams' work piles up and overlaps
                loop.x = {n: t.cuda(non_blocking=True) for n, t in steps[i][s].items()}
                got[i].append([t.clone() for t in loop.call()[2:]])
    torch.cuda.synchronize()
    for i, loop in enumerate(loops):
        table, lens, held, pos = loop.table, loop.lens, loop.held, 0
        for x, (acc, tok) in zip(steps[i], got[i]):
            table, lens, held, pos, starts, ids, positions, _, st = S.map_tokens(table, lens, held, x["new"].tolist(), loop.free,
                                                                                 pos, PAGE, B * (T + 1))
            assert st == 0
            loop.o.write(H.np_bits(x["k"]), H.np_bits(x["v"]), ids, positions)
            w_acc, w_tok, lens, gaps, _ = S.verify_step(x["target"].numpy(), x["draft"].numpy(), x["drafts"].numpy(), None,
                                                        x["uniform"].numpy(), starts, lens)
            assert min(gaps) > 2.0 ** -44 and acc.tolist() == w_acc and tok.tolist() == w_tok
        assert loop.d_lens.tolist() == lens and (loop.c.records.cpu().numpy() == loop.o.records).all()
        assert int(loop.status) == 0
