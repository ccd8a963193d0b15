"""Plain CPU restatement, in float64 and Python integers, of the operators of a serving step around the 4-bit paged
cache: attention of a ragged batch of new tokens, sampling, and forking, releasing and compacting pages.

TEST INFRASTRUCTURE, like zf_oracle.py: written from the definitions in include/zf.h, one request, row or page at a
time; the product path never imports it and it imports nothing from that path.
"""
from __future__ import annotations

import math

import numpy as np

DEV_BAD_PAGE_ID, DEV_BAD_SEQ_LEN, DEV_CAPACITY, DEV_BAD_PROBS, DEV_BAD_FORK = 0x1, 0x8, 0x100, 0x400, 0x800


# ------------------------------------------------------------------------------- chunk attention
def chunk_attention(q, k, v, pos0, scale, window=0, softcap=0.0, slopes=None, seen=None):
    """One request.  q [T][Hq][128] at positions pos0 .., k and v [L][Hkv][128], all float64; seen [L]: tokens that are
    not skipped.  Returns out, lse, and two bounds per (row, head): of |weights . |v||, of sum |v| over what is seen,
    and of the largest scale * sum |q k|."""
    T, hq, d = q.shape
    L, hkv = k.shape[:2]
    group = hq // hkv
    out, lse = np.zeros((T, hq, d)), np.full((T, hq), -math.inf)
    wv, sv, mag = np.zeros((T, hq, d)), np.zeros((T, hq, d)), np.zeros((T, hq))
    for t in range(T):
        p = pos0 + t
        j = np.arange(max(0, p - window + 1) if window else 0, min(p + 1, L))
        if seen is not None:
            j = j[seen[j]]
        if p < 0 or j.size == 0:
            continue
        for h in range(hq):
            kk, vv = k[j, h // group], v[j, h // group]
            x = scale * (kk @ q[t, h])
            mag[t, h] = (abs(scale) * (np.abs(kk) @ np.abs(q[t, h]))).max()
            if softcap:
                x = softcap * np.tanh(x / softcap)
            if slopes is not None:
                x = x + slopes[h] * (j - p)
            top = x.max()
            w = np.exp(x - top)
            out[t, h] = w @ vv / w.sum()
            wv[t, h] = w @ np.abs(vv) / w.sum()
            sv[t, h] = np.abs(vv).sum(0)
            lse[t, h] = top + math.log(w.sum())
    return out, lse, wv, sv, mag


# ------------------------------------------------------------------------------------- sampling
def sample(x, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """The kept distribution of one row of logits (float64 values): weights [V] (0: not kept), or None for a row that
    cannot be sampled from."""
    x = np.where(np.isnan(x), -math.inf, x)
    top = x.max()
    if not np.isfinite(top) or not 0 <= temperature < math.inf or top_k < 0 or not top_p >= 0 or not min_p <= 1:
        return None
    n = x.size
    if temperature < np.float32(1e-6):
        top_k, temperature, top_p, min_p = 1, 1.0, 1.0, 0.0
    with np.errstate(over="ignore"):
        w = np.exp((x - top) / float(temperature))
    order = np.argsort(-x, kind="stable")
    if top_k:
        n = min(n, top_k)
    head = w[order[:n]]
    if min_p > 0:
        n = min(n, int((head >= min_p).sum()))
        head = head[:n]
    if top_p < 1:
        run = np.cumsum(head)
        n = min(n, int((run < float(top_p) * run[-1]).sum()) + 1)
    kept = np.zeros_like(w)
    kept[order[:n]] = w[order[:n]]
    return kept


def draw(kept, u, slack=2.0 ** -28):
    """(token, tokens that a point within slack of the drawn one gives: running sums ascend, so all kept ones between
    those of its ends)."""
    run = np.cumsum(kept)
    live = np.flatnonzero(kept)
    at = lambda z: int(min(np.searchsorted(run, z, side="right"), live[-1]))  # noqa: E731
    lo, hi = at(max(0.0, u - slack) * run[-1]), at((u + slack) * run[-1])
    return at(u * run[-1]), {int(i) for i in live if lo <= i <= hi}


# ---------------------------------------------------------------------------------------- pages
def fork(table, lens, held, src, dst, free, pos, page):
    """Returns (table, lens, held, pos, copy_src, copy_dst, status); inputs are left alone."""
    B, max_pages = table.shape
    out, new_lens, new_held, status = table.copy(), list(lens), list(held), 0
    plan, named = [], set()
    for s, d in zip(src, dst):
        fresh = d not in named
        if 0 <= d < B:
            named.add(d)
        ok = 0 <= s < B and 0 <= d < B and s != d and fresh and held[d] == 0 and lens[d] == 0 and \
            0 <= held[s] <= max_pages and 0 <= lens[s] <= held[s] * page
        plan.append((s, d) if ok else None)
        if not ok:
            status |= DEV_BAD_FORK
    need = sum(1 for p in plan if p and lens[p[0]] % page)
    if pos < 0 or pos + need > len(free):
        return out, new_lens, new_held, pos, [-1] * len(src), [-1] * len(src), status | DEV_CAPACITY
    copy_src, copy_dst = [], []
    for p in plan:
        a = b = -1
        if p:
            s, d = p
            full = lens[s] // page
            out[d, :full] = table[s, :full]
            new_lens[d], new_held[d] = lens[s], full
            if lens[s] % page:
                a, b = int(table[s, full]), int(free[pos])
                out[d, full] = b
                new_held[d] += 1
                pos += 1
        copy_src.append(a)
        copy_dst.append(b)
    return out, new_lens, new_held, pos, copy_src, copy_dst, status


def release(table, lens, held, gone, free, pos, pool):
    """Returns (lens, held, free, pos, status)."""
    status = 0
    n = []
    for h in held:
        if not 0 <= h <= table.shape[1]:
            status |= DEV_BAD_SEQ_LEN
        n.append(min(max(h, 0), table.shape[1]))
    stays, freed = set(), []
    for b in range(len(n)):
        if not gone[b]:
            stays.update(int(p) for p in table[b, :n[b]])
    for b in range(len(n)):
        for p in table[b, :n[b]]:
            if not 0 <= p < pool:
                status |= DEV_BAD_PAGE_ID
            elif gone[b] and int(p) not in stays and int(p) not in freed:
                freed.append(int(p))
    if pos > len(free) or len(freed) > pos:
        return list(lens), list(held), list(free), pos, status | DEV_CAPACITY
    free = list(free)
    free[pos - len(freed):pos] = freed
    return ([0 if g else x for x, g in zip(lens, gone)], [0 if g else x for x, g in zip(held, gone)], free,
            pos - len(freed), status)


def compact(table, held, pool):
    """Returns (table, free, pos, copy_src, copy_dst, status)."""
    status, n = 0, []
    for h in held:
        if not 0 <= h <= table.shape[1]:
            status |= DEV_BAD_SEQ_LEN
        n.append(min(max(h, 0), table.shape[1]))
    used = set()
    for b, h in enumerate(n):
        for p in table[b, :h]:
            if 0 <= p < pool:
                used.add(int(p))
            else:
                status |= DEV_BAD_PAGE_ID
    k = len(used)
    moves = sorted(p for p in used if p >= k)
    holes = [p for p in range(k) if p not in used]
    to = dict(zip(moves, holes))
    out = table.copy()
    for b, h in enumerate(n):
        for j in range(h):
            out[b, j] = to.get(int(table[b, j]), table[b, j])
    pad = [-1] * (pool // 2 - len(moves))
    return out, [i if i >= k else -1 for i in range(pool)], k, moves + pad, holes + pad, status
