"""Plain CPU restatement, in float64 and Python integers, of the operators of a speculative decode step:
the 4-bit paged cache (numbers and record layout), attention over it, the slot map of new tokens and the
verification of drafted tokens.

TEST INFRASTRUCTURE, like zf_oracle.py: written from the definitions in include/zf.h, one value, token
or request at a time; the product path never imports it and it imports nothing from that path.
"""
from __future__ import annotations

import math

import numpy as np

HEAD_DIM, BLOCK, TILE, RECORD = 128, 16, 16, 2304
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# the positive e4m3 numbers, by their byte (0x7f is not one of them)
E4M3 = np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:127])

DEV_BAD_PAGE_ID, DEV_BAD_N_VALID, DEV_BAD_SEQ_LEN = 0x1, 0x4, 0x8
DEV_NOT_FINITE, DEV_CAPACITY, DEV_BAD_DRAFT, DEV_BAD_PROBS = 0x80, 0x100, 0x200, 0x400


def nearest_even(grid: np.ndarray, x: float) -> int:
    """Index of the number of an ascending grid nearest to x; of two equally near ones the even index
    (in both formats the index of a number is its bit pattern, so that is the even one)."""
    i = int(np.searchsorted(grid, x))
    if i == 0:
        return 0
    if i == len(grid):
        return len(grid) - 1
    lo, hi = x - grid[i - 1], grid[i] - x
    return i - 1 if lo < hi or (lo == hi and (i - 1) % 2 == 0) else i


def bf16_to_f64(bits: np.ndarray) -> np.ndarray:
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def f64_to_bf16(x: np.ndarray) -> np.ndarray:
    """Nearest-even BF16 bits of finite values (float32 first: exact for what is stored here)."""
    u = x.astype(np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def quantise_block(bits: np.ndarray, scale: float = 1.0):
    """16 BF16 values -> (16 codes, scale byte, whether one was not finite)."""
    x = bf16_to_f64(bits)
    odd = not np.isfinite(x).all()
    inv = np.float32(1.0) / np.float32(scale)
    with np.errstate(over="ignore", invalid="ignore"):
        t = (x.astype(np.float32) * inv).astype(np.float64)
    t[np.isnan(t)] = 0.0
    a = np.abs(t).max()
    if a == 0:
        return np.zeros(BLOCK, np.uint8), 0, odd
    want = min(max(float(np.float32(a) / np.float32(6.0)) if np.isfinite(a) else math.inf, E4M3[1]), 448.0)
    byte = nearest_even(E4M3, want)
    codes = [nearest_even(E2M1, abs(v) / E4M3[byte]) + (8 if v < 0 else 0) for v in t]
    return np.array(codes, np.uint8), byte, odd


def k_code_at(tok, byte):
    return 64 * tok + byte


def v_code_at(tok, byte):
    return 1024 + 64 * tok + (byte ^ (32 if tok & 2 else 0))


def k_scale_at(tok, block):
    return 2048 + 16 * (tok % 8) + 4 * (block // 2) + 2 * (tok // 8) + block % 2


def v_scale_at(tok, block):
    return 2176 + 16 * block + 4 * (tok % 8 // 2) + 2 * (tok // 8) + tok % 2


class Q4Cache:
    def __init__(self, num_pages, num_kv_heads, page_size, k_scale=1.0, v_scale=1.0):
        self.num_pages, self.hkv, self.page_size = num_pages, num_kv_heads, page_size
        self.k_scale, self.v_scale = k_scale, v_scale
        self.records = np.zeros((num_pages, num_kv_heads, page_size // TILE, RECORD), np.uint8)
        self.status = 0

    def write(self, k_bits, v_bits, page_ids, positions):
        """Tokens [n][hkv][128] into their places."""
        for i, (pid, pos) in enumerate(zip(page_ids, positions)):
            if pos == -1:
                continue
            if not 0 <= pid < self.num_pages:
                self.status |= DEV_BAD_PAGE_ID
                continue
            if not 0 <= pos < self.page_size:
                self.status |= DEV_BAD_N_VALID
                continue
            for h in range(self.hkv):
                rec, tok = self.records[pid, h, pos // TILE], pos % TILE
                for bits, scale, code_at, scale_at in ((k_bits, self.k_scale, k_code_at, k_scale_at),
                                                       (v_bits, self.v_scale, v_code_at, v_scale_at)):
                    for c in range(HEAD_DIM // BLOCK):
                        codes, byte, odd = quantise_block(bits[i, h, c * BLOCK:(c + 1) * BLOCK], scale)
                        self.status |= DEV_NOT_FINITE if odd else 0
                        rec[scale_at(tok, c)] = byte
                        for j in range(BLOCK // 2):
                            rec[code_at(tok, c * 8 + j)] = codes[2 * j] | codes[2 * j + 1] << 4

    def token(self, pid, h, pos):
        """(k, v) float64 [128] stored at a place."""
        rec, tok = self.records[pid, h, pos // TILE], pos % TILE
        out = []
        for scale, code_at, scale_at in ((self.k_scale, k_code_at, k_scale_at), (self.v_scale, v_code_at, v_scale_at)):
            at = np.array([code_at(tok, j) for j in range(64)])
            codes = np.stack((rec[at] & 15, rec[at] >> 4), 1).reshape(-1)
            s = E4M3[np.array([rec[scale_at(tok, c)] & 0x7F for c in range(8)])]
            x = E2M1[codes & 7] * np.where(codes > 7, -1.0, 1.0) * np.repeat(s, BLOCK)
            out.append(x * float(np.float32(scale)))
        return out


def attention(cache: Q4Cache, q_bits, table, lens, scale):
    """q_bits [B][T][Hq][128] -> (out [B][T][Hq][128], lse [B][T][Hq], bound [B][T][Hq]) in float64.
    bound: how far a float32 computation with exact operands may be off, relative to the largest
    |v|: 16 roundings of 2^-23 in each score (8 instructions of 16 products), twice for the weights and
    their sum; (n / 8 + 32) in the second product (two instructions per 16 tokens, the merges); 2^-21
    for exponentials and divisions."""
    B, T, hq, _ = q_bits.shape
    out = np.zeros((B, T, hq, HEAD_DIM))
    lse = np.full((B, T, hq), -np.inf)
    bound = np.zeros((B, T, hq))
    group = hq // cache.hkv
    for b in range(B):
        places = [(table[b, p // cache.page_size], p % cache.page_size) for p in range(lens[b])]
        good = np.array([0 <= pid < cache.num_pages for pid, _ in places], bool)
        for h in range(cache.hkv):
            kv = [cache.token(pid, h, pos) if ok else (np.zeros(HEAD_DIM),) * 2 for (pid, pos), ok in zip(places, good)]
            if not kv:
                continue
            k, v = np.array([x[0] for x in kv]), np.array([x[1] for x in kv])
            for t in range(T):
                n = lens[b] - T + t + 1
                if n <= 0 or not good[:n].any():
                    continue
                for g in range(h * group, (h + 1) * group):
                    q = bf16_to_f64(q_bits[b, t, g])
                    s = np.where(good[:n], (k[:n] @ q) * scale, -np.inf)
                    top = s.max()
                    p = np.exp(s - top)
                    lse[b, t, g] = top + math.log(p.sum())
                    out[b, t, g] = (p @ v[:n]) / p.sum()
                    size = (np.abs(k[:n]) @ np.abs(q)).max() * abs(scale)
                    bound[b, t, g] = (2 * 16 * size + n / 8 + 32 + 4) * 2.0 ** -23
    return out, lse, bound


def map_tokens(table, lens, held, new, free, free_pos, page_size, max_tokens):
    """(table, lens, held, free_pos, starts, page_ids, positions, seq_positions, status), lists and ints."""
    table, lens, held = [list(r) for r in table], list(lens), list(held)
    max_pages = len(table[0]) if table else 0
    status, plan = 0, []
    for b in range(len(lens)):
        ok = lens[b] >= 0 and new[b] >= 0 and 0 <= held[b] <= max_pages and lens[b] <= held[b] * page_size and \
            lens[b] + new[b] <= max_pages * page_size
        status |= 0 if ok else DEV_BAD_SEQ_LEN
        n = new[b] if ok else 0
        plan.append((n, max(0, -(-(lens[b] + n) // page_size) - held[b]) if ok else 0))
    if sum(n for n, _ in plan) > max_tokens or free_pos < 0 or sum(e for _, e in plan) + free_pos > len(free):
        status |= DEV_CAPACITY
        plan = [(0, 0)] * len(plan)
    starts, ids, pos, seq = [], [], [], []
    for b, (n, extra) in enumerate(plan):
        starts.append(len(ids))
        for _ in range(extra):
            table[b][held[b]] = free[free_pos]
            held[b] += 1
            free_pos += 1
        for p in range(lens[b], lens[b] + n):
            ids.append(table[b][p // page_size])
            pos.append(p % page_size)
            seq.append(p)
        lens[b] += n
    starts.append(len(ids))
    pad = [-1] * (max_tokens - len(ids))
    return table, lens, held, free_pos, starts, ids + pad, pos + pad, seq + pad, status


def verify(target, draft, drafts, n_drafts, uniform):
    """(accepted [B], tokens [B][T+1], gap [B], status): gap is how far the drawn point lies from the
    nearest border between tokens, relative to the sum of the weights."""
    B, T = drafts.shape
    V = target.shape[2]
    accepted, tokens, gaps, status = [], [], [], 0
    for b in range(B):
        n = T if n_drafts is None else int(n_drafts[b])
        if not 0 <= n <= T:
            status |= DEV_BAD_DRAFT
            n = min(max(n, 0), T)
        a = 0
        while a < n:
            x = int(drafts[b, a])
            if not 0 <= x < V:
                status |= DEV_BAD_DRAFT
                break
            q = np.float32(1.0) if draft is None else draft[b, a, x]
            if not np.float32(uniform[b, a]) * q < target[b, a, x]:
                break
            a += 1
        for _ in range(2):
            w = target[b, a].astype(np.float32).copy()
            if a < n and len(gaps) == b:
                if draft is not None:
                    w = w - draft[b, a]
                elif 0 <= drafts[b, a] < V:
                    w[drafts[b, a]] -= np.float32(1.0)
            w = np.where(w > 0, w, 0).astype(np.float64)
            if w.sum() != 0:
                break
            if len(gaps) == b:
                gaps.append(None)             # second time round: p itself
        del gaps[b:]
        total = math.fsum(w) if np.isfinite(w).all() else math.inf
        if not 0 < total < math.inf:
            token, gap = -1, math.inf
            status |= DEV_BAD_PROBS
        else:
            c = np.cumsum(w)
            r = float(np.float32(uniform[b, T])) * total
            hits = np.nonzero((c > r) & (w > 0))[0]
            token = int(hits[0]) if len(hits) else int(np.nonzero(w)[0][-1])
            gap = float(np.abs(c - r).min() / total)
        accepted.append(a)
        tokens.append([int(x) for x in drafts[b, :a]] + [token] + [-1] * (T - a))
        gaps.append(gap)
    return accepted, tokens, gaps, status


def verify_step(target, draft, drafts, n_drafts, uniform, starts, lens):
    """verify after map_tokens in one step: starts are its list starts, lens the lengths it gave.
    (accepted, tokens, lens, gaps, status); a request without places keeps its length, any other ends with
    its last token and the accepted drafts."""
    B, T = drafts.shape
    accepted, tokens, after, gaps, status = [], [], [], [], 0
    for b in range(B):
        places = int(starts[b + 1]) - int(starts[b])
        if not 1 <= places <= T + 1:
            status |= DEV_BAD_DRAFT if places else 0
            accepted.append(0)
            tokens.append([-1] * (T + 1))
            after.append(int(lens[b]))
            gaps.append(math.inf)
            continue
        n = places - 1 if n_drafts is None else int(n_drafts[b])
        if not 0 <= n <= places - 1:
            status |= DEV_BAD_DRAFT
            n = min(max(n, 0), places - 1)
        a, t, g, st = verify(target[b:b + 1], None if draft is None else draft[b:b + 1], drafts[b:b + 1], [n], uniform[b:b + 1])
        left = int(lens[b]) - (places - 1 - a[0])
        status |= st | (DEV_BAD_SEQ_LEN if left < 0 else 0)
        accepted.append(a[0])
        tokens.append(t[0])
        after.append(max(left, 0))
        gaps.append(g[0])
    return accepted, tokens, after, gaps, status
