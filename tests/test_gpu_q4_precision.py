"""How exactly the 4-bit attention computes, per instance of its kernel, with bounds from the number of roundings
(q4_precision.py)."""
import math

import numpy as np
import pytest
import torch

from oracle import zf_step_oracle as S
from tests import helpers as H
from tests import q4_precision as P

pytestmark = pytest.mark.gpu

SCALE = 1 / math.sqrt(128)


@pytest.fixture(scope="module")
def zf():
    return H.zf_module()


def filled(zf, pages, hkv, page, seed):
    """A cache whose pages are full (K normal, V positive) and its float64 contents [page][hkv][token][128]."""
    rng = np.random.default_rng(seed)
    n = pages * page
    k = torch.from_numpy(rng.standard_normal((n, hkv, 128))).to(torch.bfloat16).view(torch.int16)
    v = torch.from_numpy(np.abs(rng.standard_normal((n, hkv, 128))) + 0.5).to(torch.bfloat16).view(torch.int16)
    c, o = zf.Q4Cache(pages, hkv, page), S.Q4Cache(pages, hkv, page)
    ids, pos = [i // page for i in range(n)], [i % page for i in range(n)]
    zf.q4_write_tokens(c, k.cuda(), v.cuda(), ids, pos)
    o.records[...] = c.records.cpu().numpy()
    kv = np.array([[[o.token(p, h, t) for t in range(page)] for h in range(hkv)] for p in range(pages)])
    return c, kv[:, :, :, 0], kv[:, :, :, 1]


# (group, T): every instance of the kernel; the last takes two passes
@pytest.mark.parametrize("group,T", [(4, 1), (1, 1), (2, 2), (7, 1), (5, 1), (3, 2), (16, 1), (8, 2), (24, 1), (7, 3), (32, 1),
                                     (7, 4), (8, 5)])
def test_one_unit(zf, group, T):
    """Contexts of 1 to 32 tokens: one or two records, one step of the kernel."""
    hkv, page, lens = 2, 16, [1, 2, 3, 5, 8, 16, 17, 31, 32]
    B, rng = len(lens), np.random.default_rng(100 * group + T)
    c, k, v = filled(zf, 2 * B, hkv, page, 200 + group)
    table = rng.permutation(2 * B).reshape(B, 2)
    ks = k[table].transpose(0, 2, 1, 3, 4).reshape(B, hkv, 2 * page, 128)
    vs = v[table].transpose(0, 2, 1, 3, 4).reshape(B, hkv, 2 * page, 128)
    q = np.zeros((B, T, hkv, group, 128), np.uint16)
    for b in range(B):
        for h in range(hkv):
            q[b, :, h] = P.queries(rng, ks[b, h, :lens[b]], T * group, SCALE).reshape(T, group, 128)
    q_dev = torch.from_numpy(q.reshape(B, T, hkv * group, 128).view(np.int16)).cuda()
    out, lse = zf.q4_decode_attn(c, q_dev, torch.tensor(table, dtype=torch.int32).cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    out, lse = out.cpu().numpy().reshape(q.shape), lse.cpu().numpy().reshape(q.shape[:-1])
    for b in range(B):
        for t in range(T):
            n = lens[b] - T + t + 1
            for h in range(hkv):
                if n <= 0:
                    assert not out[b, t, h].any() and np.isneginf(lse[b, t, h]).all()
                    continue
                ref, ref_lse = P.attend(ks[b, h, :n], vs[b, h, :n], q[b, t, h], SCALE)
                off = np.abs(out[b, t, h] - ref).max() / vs[b, h, :n].max()
                assert off <= P.ONE_UNIT, (b, t, h, off / P.ONE_UNIT)
                assert np.abs(lse[b, t, h] - ref_lse).max() <= P.ONE_UNIT_LSE, (b, t, h)
    assert c.status_word() == 0


def ranges_of(group):
    """Ranges of a call that fills the device: one per warp."""
    warps = 16 if group <= 8 else 12 if group <= 16 else 8
    return torch.cuda.get_device_properties(0).multi_processor_count * warps


@pytest.mark.parametrize("group", [4, 7, 16, 24, 32])
def test_hundreds_of_millions_of_tokens(zf, group):
    """A context that repeats 32 pages, ranges of 4000 units: its result is that of the pages attended once.  The
    weights and the units' sums repeat, so their additions err alike."""
    pages, page, units = 32, 128, 4000
    c, k, v = filled(zf, pages, 1, page, 300 + group)
    k, v = k.reshape(-1, 128), v.reshape(-1, 128)
    times = -(-2 * units * ranges_of(group) // (pages * page // 16))              # 2 records a unit
    n = times * pages * page
    assert n < 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(1)
    table = torch.rand(times, pages, device="cuda", generator=g).argsort(1).to(torch.int32).view(1, -1)
    rng = np.random.default_rng(group)
    q = P.queries(rng, k, group, SCALE)
    out, lse = zf.q4_decode_attn(c, torch.from_numpy(q.view(np.int16))[None].cuda(), table,
                                 torch.tensor([n], dtype=torch.int32, device="cuda"))
    ref, ref_lse = P.attend(k, v, q, SCALE)
    units = n / 32 / ranges_of(group)
    scores = S.bf16_to_f64(q) @ k.T
    # four additions per lane and unit to the denominator, one to the result (4 units a page); 168 of the merge in
    # each, off by u of the running sum at most, half of the final one on the average
    den = max(P.repeated(4 * units, np.unique(row, return_counts=True)[1] / row.size) for row in scores) + 84 * P.U24
    num = P.repeated(units, np.full(4 * pages, 1 / (4 * pages))) + 84 * P.U24
    off = np.abs(out[0].cpu().numpy() - ref).max() / v.max()
    assert off <= P.ONE_UNIT + den + num, off / P.U24
    # the logarithm (a step at 16 to 32 and half of one) and two roundings of a value near 20
    off = np.abs(lse[0].cpu().numpy() - ref_lse - math.log(times)).max()
    assert off <= P.ONE_UNIT_LSE + den + (0.7 * 48 + 2 * 22) * P.U24, off / P.U24
    assert c.status_word() == 0


def decode(rec, code_at, scale_at):
    """Records [...][2304] -> float64 [... * 16][128] by the layout's address functions, on their device."""
    dev = rec.device
    codes = torch.tensor([[code_at(t, i) for i in range(64)] for t in range(16)], device=dev)
    scales = torch.tensor([[scale_at(t, b) for b in range(8)] for t in range(16)], device=dev)
    value = torch.tensor(np.concatenate((S.E2M1, -S.E2M1)), device=dev)
    step = torch.tensor(np.append(S.E4M3, 480.0), device=dev)
    byte = rec[..., codes].long()
    x = torch.stack((value[byte & 15], value[byte >> 4]), -1).flatten(-2)
    x = x * step[(rec[..., scales] & 0x7F).long()].repeat_interleave(16, -1)
    return x.reshape(-1, 128)


@pytest.mark.parametrize("group,units", [(4, 1500), (7, 1000), (28, 1000)])
def test_sums_of_a_long_range_are_rounded(zf, group, units):
    """One context, whose weights all differ, in ranges of 1000 units and more; V between 4 and 6.  Sums cut off
    instead would be off by 900 (4 columns: 0.72 u of the result, 5/6 of the largest V, per unit), 1200 and
    1200 u; the bounds are 318 (4 columns) and 294."""
    page = 128
    pages = units * 32 * ranges_of(group) // page
    c = zf.Q4Cache(pages, 1, page)
    g = torch.Generator(device="cuda").manual_seed(group)

    def draw(at, n, low, high, keep=0xFF, add=0):
        part = c.records[..., at:at + n]
        for i in range(0, pages, 65536):
            x = torch.randint(low, high, part[i:i + 65536].shape, dtype=torch.uint8, device="cuda", generator=g)
            part[i:i + 65536] = (x & keep) | add
    draw(0, 1024, 0, 256)                               # K: any codes
    draw(1024, 1024, 0, 256, 0x11, 0x66)                # V: 4 or 6
    draw(2048, 128, 0x30, 0x38)                         # K scales 0.5 to 0.9375
    draw(2176, 128, 0x38, 0x39)                         # V scales 1
    q = P.queries(np.random.default_rng(group), np.full((1, 128), 6 * 0.9375), group, SCALE, 4)
    n = pages * page
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, -1)
    out, lse = zf.q4_decode_attn(c, torch.from_numpy(q.view(np.int16))[None].cuda(), table,
                                 torch.tensor([n], dtype=torch.int32, device="cuda"))
    assert c.status_word() == 0
    qd = torch.tensor(S.bf16_to_f64(q) * SCALE, device="cuda")
    num, den = torch.zeros(group, 128, dtype=torch.float64, device="cuda"), torch.zeros(group, dtype=torch.float64, device="cuda")
    for i in range(0, pages, 2048):
        rec = c.records[i:i + 2048]
        p = torch.exp(decode(rec, S.k_code_at, S.k_scale_at) @ qd.T)
        num += p.T @ decode(rec, S.v_code_at, S.v_scale_at)
        den += p.sum(0)
    # a score is a sum of four products of at most half a log2 unit: eight terms cut off at 24 bits of 2, times ln 2
    bound = P.chain(units) + 2 * 11.1 * P.U24
    off = (out[0] - num / den[:, None]).abs().max().item() / 6
    assert off <= bound, off / P.U24
    off = (lse[0] - den.log()).abs().max().item()
    assert off <= bound + (0.7 * 48 + 2 * 22) * P.U24, off / P.U24
