"""The 4-bit cache, slot-map and verification kernels start before the kernel ahead of them has ended; whatever that
kernel writes late they have to see.  A helper lets the next grid start at once and writes a call's inputs
200 us later, over valid ones that would give other results."""
import math

import numpy as np
import pytest
import torch

from oracle import zf_step_oracle as S
from tests import helpers as H
from tests.test_gpu_q4 import bits, build, check, tokens
from tests.test_gpu_step import i32, map_case, same_map

pytestmark = pytest.mark.gpu

DELAY_NS = 200_000


@pytest.fixture(scope="module")
def zf():
    return H.zf_module()


def late(call, *pairs):
    """`call` right behind a kernel that copies each (new, live) pair of device tensors 200 us after the call may
    start.  A third pair and more are copied by a kernel before that one."""
    late_copy, stream = H.late_writer(), torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    pairs = [(n.contiguous(), live) for n, live in pairs]
    for n, live in pairs:
        assert n.dtype == live.dtype and n.shape == live.shape and live.is_contiguous()
    groups = [pairs[i:i + 2] for i in range(0, len(pairs), 2)]
    for g in groups:
        args = []
        for n, live in g + [(None, None)] * (2 - len(g)):
            args += [n.data_ptr(), live.data_ptr(), n.numel() * n.element_size() // 4] if n is not None else [None, None, 0]
        assert late_copy(*args, DELAY_NS, stream) == 0
    out = call()
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("what", ["places", "values"])
def test_write_sees_what_is_written_late(zf, what):
    n, hkv, page, pool = 64, 2, 32, 4
    k, v = tokens(n, hkv, 1)
    k0, v0 = tokens(n, hkv, 2)
    at = np.random.default_rng(3).permutation(pool * page)
    ids, pos = i32(at[:n] // page), i32(at[:n] % page)
    ids0, pos0 = i32(at[n:] // page), i32(at[n:] % page)
    if what == "places":
        k0, v0 = k, v
    else:
        ids0, pos0 = ids, pos
    c, o = zf.Q4Cache(pool, hkv, page), S.Q4Cache(pool, hkv, page)
    live = [t.cuda() for t in (ids0, pos0, k0, v0)]
    new = [t.cuda() for t in (ids, pos, k, v)]
    pick = (0, 1) if what == "places" else (2, 3)
    late(lambda: zf.q4_write_tokens(c, live[2], live[3], live[0], live[1]), *[(new[i], live[i]) for i in pick])
    o.write(H.np_bits(k), H.np_bits(v), ids.tolist(), pos.tolist())
    assert (c.records.cpu().numpy() == o.records).all() and c.status_word() == 0


@pytest.mark.parametrize("what", ["places", "records"])
def test_read_sees_what_is_written_late(zf, what):
    n, hkv, page, pool = 64, 2, 32, 4
    k, v = tokens(pool * page, hkv, 4)
    c, o = zf.Q4Cache(pool, hkv, page), S.Q4Cache(pool, hkv, page)
    every = [i // page for i in range(pool * page)], [i % page for i in range(pool * page)]
    o.write(H.np_bits(k), H.np_bits(v), *every)
    at = np.random.default_rng(5).permutation(pool * page)
    ids, pos = i32(at[:n] // page).cuda(), i32(at[:n] % page).cuda()
    good = torch.from_numpy(o.records).cuda()
    if what == "places":
        c.records.copy_(good)
        ids0, pos0 = i32(at[n:] // page).cuda(), i32(at[n:] % page).cuda()
        kr, vr = late(lambda: zf.q4_read_tokens(c, ids0, pos0), (ids, ids0), (pos, pos0))
    else:
        kr, vr = late(lambda: zf.q4_read_tokens(c, ids, pos), (good, c.records))
    for i in range(n):
        ek, ev = o.token(int(ids[i]), 1, int(pos[i]))
        assert (S.bf16_to_f64(H.np_bits(kr[i, 1])) == ek).all() and (S.bf16_to_f64(H.np_bits(vr[i, 1])) == ev).all()


# (group, T): an instance of the kernel each
INSTANCES = [(4, 1), (2, 2), (7, 1), (3, 2), (8, 2), (7, 3), (7, 4)]


@pytest.mark.parametrize("group,T", INSTANCES)
def test_attention_sees_what_is_written_late(zf, group, T):
    lens, hkv, page = [700, 33, 130], 2, 16
    c, o, table, sl = build(zf, lens, hkv, page, 31)
    g = torch.Generator().manual_seed(32)
    qs = [bits(torch.randn(3, T, hkv * group, 128, generator=g)) for _ in range(4)]
    table2, lens2 = table.flip(0).contiguous(), [130, 20, 600]
    live = [t.cuda() for t in (qs[0], table, sl)]
    records = c.records.clone()
    ws = zf.new_workspace(zf.q4_workspace_size(3, T, hkv * group, hkv, page, table.shape[1]))

    def call():
        return zf.q4_decode_attn(c, *live, workspace=ws)

    def right(res, q, t, L):
        ref, ref_lse, bound = S.attention(o, H.np_bits(q), t.numpy(), L, 1 / math.sqrt(128))
        check(*res, ref, ref_lse, bound, 6.0, bound)
        assert c.status_word() == 0
    right(call(), qs[0], table, lens)
    # the queries, in the buffer that the calls before have read
    for q in qs[1:]:
        right(late(call, (q.cuda(), live[0])), q, table, lens)
    right(late(call, (table2.cuda(), live[1]), (i32(lens2).cuda(), live[2])), qs[3], table2, lens2)
    # the cache's records (only zeros before)
    c.records.zero_()
    right(late(call, (records, c.records)), qs[3], table2, lens2)


@pytest.mark.parametrize("B,max_pages,new_max,most", [(40, 12, 20, 4096), (40, 60, 300, 32768), (40, 60, 300, 50000)])
def test_map_sees_what_is_written_late(zf, B, max_pages, new_max, most):
    """One CTA, a cluster of 8, and the second kernel of long lists."""
    table, lens, held, new, free = map_case(B, 16, max_pages, new_max, 6)
    assert int(new.sum()) <= most
    want = S.map_tokens(table, lens, held, new, free, 2, 16, most)
    assert want[-1] == 0
    good = [i32(x).cuda() for x in (table, lens, held, new, free, [2])]
    for pick in ((1, 3), (2, 5), (0, 4)):
        live = [t.clone() for t in good]
        live[0 if 0 in pick else 5].fill_(0) if pick != (1, 3) else live[3].fill_(1)
        if 1 in pick:
            live[1].zero_()
        if 2 in pick:
            live[2].fill_(max_pages)
        if 4 in pick:
            live[4].copy_(good[4].flip(0))
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        m = late(lambda: zf.map_tokens(*live, 16, most, status=status), *[(good[i], live[i]) for i in pick])
        same_map(live[0], m, int(status), want)


@pytest.mark.parametrize("B,V", [(3, 900), (3, 20001), (300, 516)])
def test_verify_sees_what_is_written_late(zf, B, V):
    T = 3
    g = torch.Generator().manual_seed(V)
    target = torch.softmax(torch.randn(B, T + 1, V, generator=g), -1)
    draft = torch.softmax(torch.randn(B, T, V, generator=g), -1)
    drafts = torch.multinomial(draft.reshape(B * T, V), 1, generator=g).view(B, T).to(torch.int32)
    uniform = torch.rand(B, T + 1, generator=g)
    n, lens = i32(np.arange(B) % (T + 1)), i32(50 + np.arange(B))
    starts = i32(np.arange(B + 1) * (T + 1))
    want = S.verify_step(target.numpy(), draft.numpy(), drafts.numpy(), n.numpy(), uniform.numpy(), starts.tolist(), lens.tolist())
    assert min(want[3]) > 2.0 ** -44 and want[4] == 0
    good = [t.cuda() for t in (target, draft, drafts, uniform, n, starts, lens)]
    old = [t.cuda() for t in (target.flip(-1).contiguous(), draft.flip(-1).contiguous(), (drafts + 1) % V, 1 - uniform,
                              T - n, torch.zeros_like(starts), lens + 9)]
    for pick in ((0, 1), (2, 3), (4, 5), (6,)):
        live = [(old if i in pick else good)[i].clone() for i in range(7)]
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        acc, tok = late(lambda: zf.verify_drafts(live[0], live[2], live[3], draft_probs=live[1], n_drafts=live[4],
                                                 seq_lens=live[6], new_seq_lens=live[6], token_start=live[5], status=status),
                        *[(good[i], live[i]) for i in pick])
        assert acc.tolist() == want[0] and tok.tolist() == want[1] and live[6].tolist() == want[2] and int(status) == 0


def test_a_step_behind_a_late_writer(zf):
    """Map, write, attend and verify in a row, each started early behind the one before, behind a kernel that writes
    the lengths and the numbers of new tokens late."""
    B, T, hkv, hq, page, V = 3, 3, 2, 8, 16, 4000
    lens = [300, 17, 95]
    c, o, table, sl = build(zf, lens, hkv, page, 33)
    held = [-(-L // page) for L in lens]
    wide = np.full((B, table.shape[1] + 3), -1)
    wide[:, :table.shape[1]] = table.numpy()
    used = set(wide[b, j] for b in range(B) for j in range(held[b]))
    free = [p for p in range(c.num_pages) if p not in used]
    g = torch.Generator().manual_seed(34)
    k, v = tokens(B * (T + 1), hkv, 35)
    q = bits(torch.randn(B, T + 1, hq, 128, generator=g))
    target = torch.softmax(torch.randn(B, T + 1, V, generator=g), -1)
    drafts, uniform = torch.randint(0, V, (B, T), generator=g).to(torch.int32), torch.rand(B, T + 1, generator=g)
    new = [T + 1, 0, T + 1]
    w_table, w_lens, w_held, w_pos, starts, ids, pos, _, st = S.map_tokens(wide, lens, held, new, free, 0, page, B * (T + 1))
    assert st == 0
    live_lens, live_new = i32([5, 5, 5]).cuda(), i32([1, 1, 1]).cuda()
    d_table, d_held, d_free, d_pos = i32(wide).cuda(), i32(held).cuda(), i32(free).cuda(), i32([0]).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lists = [torch.empty(B * (T + 1), dtype=torch.int32, device="cuda") for _ in range(3)]
    out = zf.TokenMap(live_lens, d_held, d_pos, torch.empty(B + 1, dtype=torch.int32, device="cuda"), *lists)
    kd, vd, qd, td, dd, ud = (t.cuda() for t in (k, v, q, target, drafts, uniform))
    ws = zf.new_workspace(zf.q4_workspace_size(B, T + 1, hq, hkv, page, wide.shape[1]))

    def call():
        m = zf.map_tokens(d_table, live_lens, d_held, live_new, d_free, d_pos, page, B * (T + 1), out=out, status=status)
        zf.q4_write_tokens(c, kd, vd, m.page_ids, m.positions)
        res = zf.q4_decode_attn(c, qd, d_table, m.seq_lens, workspace=ws)
        return res, zf.verify_drafts(td, dd, ud, seq_lens=live_lens, new_seq_lens=live_lens, token_start=m.token_start,
                                     status=status)
    (o4, l4), (acc, tok) = late(call, (i32(lens).cuda(), live_lens), (i32(new).cuda(), live_new))
    o.write(H.np_bits(k), H.np_bits(v), ids, pos)
    assert d_table.cpu().tolist() == [list(map(int, r)) for r in w_table] and (c.records.cpu().numpy() == o.records).all()
    ref, ref_lse, bound = S.attention(o, H.np_bits(q), np.array(w_table), w_lens, 1 / math.sqrt(128))
    check(o4, l4, ref, ref_lse, bound, 6.0, bound)
    want = S.verify_step(target.numpy(), None, drafts.numpy(), None, uniform.numpy(), starts, w_lens)
    assert min(want[3]) > 2.0 ** -44
    assert acc.tolist() == want[0] and tok.tolist() == want[1] and live_lens.tolist() == want[2]
    assert int(status) == want[4] == 0 and c.status_word() == 0
