"""Measured cases of the operators around the 4-bit paged cache that a serving step needs besides decode.

chunk    zf_q4_chunk_attn: attention of a ragged batch of new tokens (prompts in chunks, single tokens, both) over
         the cache, with a window, capped scores or a bias that grows with the distance
sample   zf_sample_tokens: temperature, top-k, min-p and top-p from given random numbers, tokens and probabilities
fork     zf_fork_requests + zf_q4_copy_pages: requests that continue another's tokens share its full pages
reclaim  zf_release_requests + zf_compact_pages + zf_q4_copy_pages: finished requests' pages, the rest moved together

`own` False runs the plain form (elementary torch operations), True the library's entry points.
"""
import math

import torch

own = False

D = 128                    # head dim
G = 16                     # channels per scale
TILE = 16                  # tokens per record
RECORD = 2304              # K codes 1024, V codes 1024, K scales 128, V scales 128
MAGS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------ the cases
def _chunk(name, **kw):
    return dict(name=name, op="chunk", window=0, softcap=0.0, slopes=False, **kw)


def listed():
    return [
        # the last 16 tokens of a prompt of the tiny configuration: latency of a short call
        _chunk("chunk_b1_t16", batch=1, hq=32, hkv=8, new_min=16, new=16, ctx_min=512, ctx=512, page=16),
        # a served step that mixes chunks of prompts with requests that decode, ragged
        _chunk("chunk_b32_mixed", batch=32, hq=32, hkv=8, new_min=1, new=512, ctx_min=512, ctx=4096, page=16),
        # an 8192-token prompt at once, one query head per kv head
        _chunk("chunk_prompt_mha", batch=1, hq=32, hkv=32, new_min=8192, new=8192, ctx_min=8192, ctx=8192, page=16),
        # a 2048-token chunk behind a long context (the long-context configuration)
        _chunk("chunk_long", batch=1, hq=32, hkv=8, new_min=2048, new=2048, ctx_min=131072, ctx=131072, page=64),
        # GQA 7, chunks of several prompts, a sliding window and capped scores
        dict(_chunk("chunk_gqa7_window_cap", batch=4, hq=28, hkv=4, new_min=1000, new=2048, ctx_min=4096, ctx=8192, page=16),
             window=4096, softcap=50.0),
        # single tokens of a served batch, scores biased by distance
        dict(_chunk("chunk_b64_t1_slopes", batch=64, hq=32, hkv=8, new_min=1, new=1, ctx_min=1024, ctx=8192, page=16),
             slopes=True),
        # a served batch, a large vocabulary, BF16 logits, every filter
        dict(name="sample_b64", op="sample", rows=64, vocab=128000, dtype="bfloat16", top_k=True, top_p=True, min_p=True,
             probs=False),
        # the distributions of 64 requests' four drafts and one more token, for their verification; odd vocabulary
        dict(name="sample_probs", op="sample", rows=320, vocab=50001, dtype="float32", top_k=False, top_p=True, min_p=False,
             probs=True),
        # four answers to each of 16 prompts
        dict(name="fork_b64", op="fork", batch=64, sources=16, forks=48, hkv=8, page=16, ctx=1024),
        # 64 continuations of one long prompt, large pages
        dict(name="fork_prefix", op="fork", batch=65, sources=1, forks=64, hkv=8, page=64, ctx=8192),
        # a few requests of a served batch are done
        dict(name="reclaim_b64", op="reclaim", batch=64, released=8, hkv=8, page=16, ctx=1024, shared=0.5),
        # most of a large batch is done, the rest is moved together
        dict(name="reclaim_b512", op="reclaim", batch=512, released=384, hkv=4, page=16, ctx=2048, shared=0.25),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk", "sample", "sample", "fork", "reclaim"])
    if op == "chunk":
        hkv = rng.choice([1, 2, 4, 8, 16, 32])
        hq = hkv * rng.randint(1, 8 if hkv < 16 else 3)
        batch = _log(rng, 1, 128)
        # at most the cache and the scores of the largest listed cases
        ctx = _log(rng, 1, max(2, min(131072, 4194304 // (batch * hkv))))
        new = _log(rng, 1, max(1, min(ctx, 8192, 8000000000 // (batch * hq * ctx))))
        return dict(op=op, batch=batch, hq=hq, hkv=hkv, new_min=rng.choice([new, 1, 0 if batch > 3 and new > 7 else 1]), new=new,
                    ctx_min=rng.choice([ctx, max(1, ctx // 8)]), ctx=ctx, page=rng.choice([16, 32, 48, 64, 128]),
                    window=rng.choice([0, 0, _log(rng, 1, 4096)]), softcap=rng.choice([0.0, 0.0, 30.0, 50.0]),
                    slopes=rng.random() < 0.25)
    if op == "sample":
        rows = _log(rng, 1, 320)
        return dict(op=op, rows=rows, vocab=_log(rng, 100, min(256000, 16000000 // rows)),
                    dtype=rng.choice(["float32", "bfloat16", "float16"]), top_k=rng.random() < 0.5, top_p=rng.random() < 0.6,
                    min_p=rng.random() < 0.3, probs=rng.random() < 0.4)
    hkv, page = rng.choice([1, 2, 4, 8, 16]), rng.choice([16, 32, 48, 64, 128])
    batch = _log(rng, 2, 512)
    ctx = _log(rng, 1, min(8192, 4000000 // (batch * hkv)))
    if op == "fork":
        sources = rng.randint(1, batch // 2)
        return dict(op=op, batch=batch, sources=sources, forks=rng.randint(1, batch - sources), hkv=hkv, page=page, ctx=ctx)
    return dict(op=op, batch=batch, released=rng.randint(0, batch), hkv=hkv, page=page, ctx=ctx, shared=rng.choice([0.0, 0.3, 0.8]))


def _seen(new, L, window):
    """Pairs of a query and a position it sees, for the last `new` of L tokens."""
    first = L - new
    full = new * first + new * (new + 1) / 2
    if not window:
        return full
    w = min(window, L)
    # the rows at positions below w - 1 see all before them, the others w
    short = max(0, min(L, w - 1) - first)
    return short * first + short * (short + 1) / 2 + (new - short) * w


def work(case):
    c = case
    if c["op"] == "chunk":
        new, L = (c["new_min"] + c["new"]) / 2, (c["ctx_min"] + c["ctx"]) / 2
        new = min(new, L)
        tokens = min(L, c["window"] + new) if c["window"] else L
        rows = c["batch"] * new * c["hq"]          # q and out in BF16, lse in float32
        return {"bytes": c["batch"] * tokens * (c["hkv"] * RECORD / TILE + 4.0 / c["page"]) + rows * (4 * D + 4) + 8.0 * c["batch"],
                "flops": 4.0 * D * c["batch"] * c["hq"] * _seen(new, L, c["window"])}
    if c["op"] == "sample":
        size = 4 if c["dtype"] == "float32" else 2
        n = float(c["rows"]) * c["vocab"]
        return {"bytes": n * (size + (4 if c["probs"] else 0)) + 24.0 * c["rows"], "flops": 4.0 * n}
    page_bytes = c["hkv"] * c["page"] // TILE * RECORD
    pages = (c["ctx"] / 2 + c["ctx"]) / 2 / c["page"]
    if c["op"] == "fork":      # the tail pages are read and written, the table's rows too
        return {"bytes": c["forks"] * (2.0 * page_bytes + 8.0 * pages + 32), "flops": 0.0}
    held = (c["batch"] - c["released"]) * pages * (1 - c["shared"])
    moved = held * c["released"] / max(c["batch"], 1)       # a page lies above the border as often as others are gone
    return {"bytes": 2.0 * page_bytes * moved + 12.0 * c["batch"] * pages, "flops": 0.0}


# ------------------------------------------------------------------------------------ the inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _kv(rows, heads, g):
    """Keys with per-channel spread and four strong channels, values N(0, 1): BF16."""
    s = torch.exp(0.5 * torch.randn(D, generator=g, device="cuda"))
    s[:4] *= 10.0
    k = torch.randn(rows, heads, D, generator=g, device="cuda") * s
    v = torch.randn(rows, heads, D, generator=g, device="cuda")
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


def _pages_of(lens, page, max_pages, pool, g):
    """Page table of `lens` tokens per request over a shuffled pool; -1 past each request's pages."""
    count = (lens + page - 1) // page
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    first = torch.cumsum(count, 0) - count
    j = torch.arange(max_pages, device="cuda")
    at = (first[:, None] + j[None]).clamp(max=pool - 1)
    return torch.where(j[None] < count[:, None], perm[at], torch.full_like(at, -1, dtype=torch.int32)), count, perm


def _bank(g):
    """A pool of quantised records, 16 tokens each."""
    k, v = _kv(2048 * TILE, 1, g)
    return _records(k.view(2048, TILE, D), v.view(2048, TILE, D))


def _rand(lo, hi, n, g):
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda")


def _spread(lo, hi, n, g):
    """n lengths from lo to hi in a random order: the same in all for every seed."""
    x = torch.linspace(lo, hi, n, dtype=torch.float64, device="cuda") if n > 1 else torch.full((1,), float(hi), device="cuda")
    return x.round().long()[torch.randperm(n, generator=g, device="cuda")]


def prepare(case, seed):
    c, g = case, _gen(seed)
    state = dict(case=c)
    if c["op"] == "chunk":
        B, page = c["batch"], c["page"]
        new = _spread(c["new_min"], c["new"], B, g)
        lens = torch.maximum(_spread(c["ctx_min"], c["ctx"], B, g), new)
        max_pages = -(-c["ctx"] // page)
        pool = int(((lens + page - 1) // page).sum()) + 1
        table, _, _ = _pages_of(lens, page, max_pages, pool, g)
        bank = _bank(g)
        pick = torch.randint(0, bank.shape[0], (pool * c["hkv"] * (page // TILE),), generator=g, device="cuda")
        start = torch.cat((torch.zeros(1, dtype=torch.long, device="cuda"), torch.cumsum(new, 0))).to(torch.int32)
        q = torch.randn(int(new.sum()), c["hq"], D, generator=g, device="cuda").to(torch.bfloat16)
        slopes = None
        if c["slopes"]:          # the usual geometric slopes, in a shuffled order
            slopes = torch.exp2(-8.0 * torch.arange(1, c["hq"] + 1, device="cuda") / c["hq"]).float()
            slopes = slopes[torch.randperm(c["hq"], generator=g, device="cuda")].contiguous()
        state.update(records=bank[pick].view(pool, c["hkv"], page // TILE, RECORD), table=table, lens=lens.to(torch.int32),
                     start=start, q=q, slopes=slopes)
    elif c["op"] == "sample":
        R, V = c["rows"], c["vocab"]
        # a few likely tokens over a broad rest
        logits = 2.0 * torch.randn(R, V, generator=g, device="cuda")
        likely = torch.randint(0, V, (R, 24), generator=g, device="cuda")
        logits.scatter_add_(1, likely, 8.0 * torch.rand(R, 24, generator=g, device="cuda"))
        logits = logits.to(getattr(torch, c["dtype"]))
        state.update(logits=logits, uniform=torch.rand(R, generator=g, device="cuda"),
                     temperature=0.5 + torch.rand(R, generator=g, device="cuda"), top_k=None, top_p=None, min_p=None)
        if c["top_k"]:           # some rows without
            k = _rand(1, 200, R, g)
            state["top_k"] = (k * (torch.rand(R, generator=g, device="cuda") < 0.8)).to(torch.int32)
        if c["top_p"]:
            state["top_p"] = 0.5 + 0.5 * torch.rand(R, generator=g, device="cuda")
        if c["min_p"]:
            state["min_p"] = 0.2 * torch.rand(R, generator=g, device="cuda")
    else:
        B, page = c["batch"], c["page"]
        max_pages = -(-c["ctx"] // page) + 1
        lens = _spread(max(1, c["ctx"] // 2), c["ctx"], B, g)
        pages = int(((lens + page - 1) // page).sum())
        order = torch.randperm(B, generator=g, device="cuda")
        if c["op"] == "fork":
            free_rows, src_rows = order[:c["forks"]], order[c["forks"]:c["forks"] + c["sources"]]
            lens[free_rows] = 0
            pool = pages + c["forks"] + 1
            table, held, perm = _pages_of(lens, page, max_pages, pool, g)
            src = src_rows[torch.arange(c["forks"], device="cuda") % c["sources"]]
            state.update(src=src.to(torch.int32), dst=free_rows.to(torch.int32), free=perm, free_pos=held.sum(dtype=torch.int32).view(1))
        else:
            count = (lens + page - 1) // page
            pool = pages + pages // 8 + 1
            table, held, perm = _pages_of(lens, page, max_pages, pool, g)
            # groups of eight requests begin with the same pages (a prompt and its forks)
            first = torch.arange(B, device="cuda") // 8 * 8
            common = (torch.minimum(count, count[first]) * c["shared"]).long()
            j = torch.arange(max_pages, device="cuda")[None]
            table = torch.where(j < common[:, None], table[first], table)
            release = torch.zeros(B, dtype=torch.int32, device="cuda")
            release[order[:c["released"]]] = 1
            # a free list over all pages: what is held lies before free_pos
            used = torch.zeros(pool, dtype=torch.bool, device="cuda")
            used[table[j < count[:, None]].long()] = True
            free = torch.cat((torch.full((int(used.sum()),), -1, dtype=torch.int32, device="cuda"),
                              torch.nonzero(~used)[:, 0].to(torch.int32)))
            state.update(release=release, free=free, free_pos=used.sum(dtype=torch.int32).view(1))
        bank = _bank(g)
        pick = torch.randint(0, bank.shape[0], (pool * c["hkv"] * (page // TILE),), generator=g, device="cuda")
        state.update(records=bank[pick].view(pool, c["hkv"], page // TILE, RECORD), table=table.contiguous(),
                     lens=lens.to(torch.int32), held=held.to(torch.int32), pool=pool)
    return _handles(state) if own else state


def _handles(state):
    """What a user's program of the library keeps: the cache object, the attention workspace, a buffer of probabilities."""
    from decode_attention_compressed_gb300 import zf
    c = state["case"]
    if c["op"] != "sample":
        state["cache"] = zf.Q4Cache(state["records"].shape[0], c["hkv"], c["page"], records=state["records"])
    if c["op"] == "chunk":
        state["workspace"] = zf.new_workspace(zf.q4_chunk_workspace_size(c["batch"], state["q"].shape[0], c["hq"], c["hkv"],
                                                                         c["page"], state["table"].shape[1]))
    if c["op"] == "sample" and c["probs"]:
        state["probs"] = torch.empty(c["rows"], c["vocab"], dtype=torch.float32, device="cuda")
    return state


# ------------------------------------------------------------------------------------ the 4-bit format, plain
def _quantise(x):
    """[..., 128] -> (codes 0..15 [..., 128], scales [..., 8] e4m3): the largest of 16 channels over 6 is
    the scale, each channel over the scale goes to the nearest of +-MAGS, ties to the even code."""
    t = x.float().unflatten(-1, (D // G, G))
    a = t.abs().amax(-1)
    s = (a / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn).float()
    s = torch.where(a > 0, s.clamp(min=2.0 ** -9), torch.zeros_like(s))
    r = t.abs() / torch.where(s > 0, s, torch.ones_like(s))[..., None]
    m = (r > 0.25).to(torch.uint8) + (r >= 0.75) + (r > 1.25) + (r >= 1.75) + (r > 2.5) + (r >= 3.5) + (r > 5.0)
    return (m + 8 * (t < 0).to(torch.uint8)).flatten(-2), s.to(torch.float8_e4m3fn)


def _pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _values(packed, scales):
    """The float32 values of packed codes [..., 64] and e4m3 scales [..., 8]."""
    table = torch.tensor(MAGS + tuple(-m for m in MAGS), device=packed.device)
    both = torch.stack((packed & 15, packed >> 4), -1).flatten(-2)
    return (table[both.int()].unflatten(-1, (D // G, G)) * scales.float()[..., None]).flatten(-2)


def _swap_halves(packed):
    """The 32-byte halves of the rows (64 packed bytes) of tokens with bit 1 set change places."""
    odd = (torch.arange(TILE, device=packed.device) & 2 > 0)[:, None]
    return torch.where(odd, packed.roll(D // 4, -1), packed)


def _records(k, v):
    """[n, 16, 128] keys and values -> [n, 2304] records.  Scale order: K byte (tok % 8) * 16 +
    (block / 2) * 4 + (tok / 8) * 2 + block % 2; V byte block * 16 + (tok % 8 / 2) * 4 + (tok / 8) * 2 + tok % 2."""
    n = k.shape[0]
    kc, ks = _quantise(k)
    vc, vs = _quantise(v)
    ks = ks.view(torch.uint8).view(n, 2, 8, 4, 2).permute(0, 2, 3, 1, 4).reshape(n, 128)
    vs = vs.view(torch.uint8).view(n, 2, 4, 2, 8).permute(0, 4, 2, 1, 3).reshape(n, 128)
    return torch.cat((_pack(kc).reshape(n, 1024), _swap_halves(_pack(vc)).reshape(n, 1024), ks, vs), 1)


def _unrecord(rec):
    """Records [..., 2304] -> float32 keys and values [..., 16, 128]."""
    lead = rec.shape[:-1]
    ks = rec[..., 2048:2176].reshape(*lead, 8, 4, 2, 2).movedim(-2, -4).reshape(*lead, 16, 8)
    vs = rec[..., 2176:2304].reshape(*lead, 8, 4, 2, 2).movedim(-4, -1).transpose(-4, -3).reshape(*lead, 16, 8)
    k = _values(rec[..., :1024].reshape(*lead, 16, 64), ks.contiguous().view(torch.float8_e4m3fn))
    v = _values(_swap_halves(rec[..., 1024:2048].reshape(*lead, 16, 64)), vs.contiguous().view(torch.float8_e4m3fn))
    return k, v


# ------------------------------------------------------------------------------------ the operators, plain
def _plain_chunk(s):
    # padded to the case's largest chunk and context; scores are worked on in place
    c, q, dev = s["case"], s["q"], s["q"].device
    B, hkv, page, group = c["batch"], c["hkv"], c["page"], c["hq"] // c["hkv"]
    start, lens = s["start"].long(), s["lens"].long()
    new, T = start[1:] - start[:-1], min(c["new"], c["ctx"])
    row = torch.arange(q.shape[0], device=dev)
    b = torch.searchsorted(start, row, right=True) - 1
    t = row - start[b]
    k, v = (x.transpose(1, 2).reshape(B, hkv, -1, D) for x in _unrecord(s["records"][s["table"].clamp(min=0).long()]))
    padded = torch.zeros(B, T, c["hq"], D, device=dev)
    padded[b, t] = q.float()
    padded = padded.view(B, T, hkv, group, D).permute(0, 2, 3, 1, 4).reshape(B, hkv, group * T, D)
    x = torch.matmul(padded, k.transpose(-1, -2)).view(B, hkv, group, T, -1).mul_(1.0 / math.sqrt(D))
    if c["softcap"]:
        x.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    pos = (lens - new)[:, None] + torch.arange(T, device=dev)[None]
    far = pos[:, :, None] - torch.arange(k.shape[2], device=dev)                          # distance back
    if s["slopes"] is not None:
        x -= s["slopes"].view(1, hkv, group, 1, 1) * far[:, None, None]
    hide = far < 0
    if c["window"]:
        hide |= far >= c["window"]
    x.masked_fill_(hide[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, hkv, group * T, -1), v).view(B, hkv, group, T, D) / total
    lse = (torch.log(total) + top)[..., 0]
    out = o.permute(0, 3, 1, 2, 4)[b, t].reshape(-1, c["hq"], D).to(torch.bfloat16)
    return out, lse.permute(0, 3, 1, 2)[b, t].reshape(-1, c["hq"])


def _plain_sample(s):
    V = s["case"]["vocab"]
    x = s["logits"].double()
    w = torch.exp((x - x.amax(-1, keepdim=True)) / s["temperature"].double()[:, None])
    keep = torch.ones_like(w, dtype=torch.bool)
    ws, order = torch.sort(w, dim=-1, descending=True, stable=True)
    if s["top_k"] is not None:
        k = torch.where(s["top_k"] > 0, s["top_k"], torch.full_like(s["top_k"], V))
        keep &= torch.arange(V, device=w.device)[None] < k[:, None]
    if s["min_p"] is not None:
        keep &= ws >= s["min_p"].double()[:, None]
    if s["top_p"] is not None:
        cum = torch.cumsum(ws * keep, -1)
        keep &= cum - ws < s["top_p"].double()[:, None] * cum[:, -1:]
    w = torch.zeros_like(w).scatter_(1, order, ws * keep)
    cum = torch.cumsum(w, -1)
    token = (cum <= s["uniform"].double()[:, None] * cum[:, -1:]).sum(-1).clamp(max=V - 1).to(torch.int32)
    return (token, (w / cum[:, -1:]).float()) if s["case"]["probs"] else token


def _plain_fork(s):
    page, lens, held, pos = s["case"]["page"], s["lens"].long(), s["held"].long(), s["free_pos"].long()
    src, dst = s["src"].long(), s["dst"].long()
    L = lens[src]
    full, tail = L // page, (L % page > 0).long()
    new = s["free"][(pos + torch.cumsum(tail, 0) - tail).clamp(max=s["free"].shape[0] - 1)]
    j = torch.arange(s["table"].shape[1], device=lens.device)[None]
    rows = torch.where(j < full[:, None], s["table"][src], s["table"][dst])
    rows = torch.where((j == full[:, None]) & (tail > 0)[:, None], new[:, None], rows)
    none = torch.full_like(new, -1)
    copy_src = torch.where(tail > 0, s["table"][src, full.clamp(max=j.shape[1] - 1)], none)
    copy_dst = torch.where(tail > 0, new, none)
    s["table"][dst] = rows
    at = tail.nonzero()[:, 0]
    s["records"][copy_dst[at].long()] = s["records"][copy_src[at].long()]
    lens[dst] = L
    held[dst] = full + tail
    return (s["table"], lens.to(torch.int32), held.to(torch.int32), (pos + tail.sum()).to(torch.int32), copy_src, copy_dst,
            s["records"])


def _plain_reclaim(s):
    dev, pool = s["table"].device, s["pool"]
    table, held, gone = s["table"].long(), s["held"].long(), s["release"] > 0
    j = torch.arange(table.shape[1], device=dev)[None]
    live = j < held[:, None]
    # pages that only finished requests hold, in the order of their first mention
    kept = torch.zeros(pool, dtype=torch.bool, device=dev)
    kept[table[live & ~gone[:, None]]] = True
    mine = table[live & gone[:, None]]
    mine = mine[~kept[mine]]
    first = torch.full((pool,), mine.shape[0], dtype=torch.long, device=dev)
    first.scatter_reduce_(0, mine, torch.arange(mine.shape[0], device=dev), "amin")
    mine = mine[first[mine] == torch.arange(mine.shape[0], device=dev)]
    pos = s["free_pos"].long()
    new_pos = pos - mine.shape[0]
    s["free"][new_pos + torch.arange(mine.shape[0], device=dev)] = mine.to(torch.int32)
    lens, held = torch.where(gone, 0, s["lens"].long()), torch.where(gone, 0, held)
    # the pages that are still held, moved to the front
    live = j < held[:, None]
    used = torch.zeros(pool, dtype=torch.bool, device=dev)
    used[table[live]] = True
    n = used.sum()
    ids = torch.arange(pool, device=dev)
    move, hole = ids[used & (ids >= n)], ids[~used & (ids < n)]
    to = ids.clone()
    to[move] = hole
    new_table = torch.where(live, to[table.clamp(min=0)], table).to(torch.int32)
    s["records"][hole] = s["records"][move]
    lists = torch.full((2, pool // 2), -1, dtype=torch.int32, device=dev)
    lists[0, :move.shape[0]] = move.to(torch.int32)
    lists[1, :move.shape[0]] = hole.to(torch.int32)
    free = torch.where(ids >= n, ids, -1).to(torch.int32)
    return (lens.to(torch.int32), held.to(torch.int32), new_pos.to(torch.int32), s["free"], new_table, free,
            n.to(torch.int32).view(1), lists[0], lists[1], s["records"])


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"chunk": _plain_chunk, "sample": _plain_sample, "fork": _plain_fork, "reclaim": _plain_reclaim}[c["op"]](s)
    from decode_attention_compressed_gb300 import zf
    if c["op"] == "chunk":
        return zf.q4_chunk_attn(s["cache"], s["q"], s["table"], s["lens"], s["start"], window=c["window"],
                                softcap=c["softcap"], slopes=s["slopes"], workspace=s["workspace"])
    if c["op"] == "sample":
        tokens = zf.sample_tokens(s["logits"], s["uniform"], temperature=s["temperature"], top_k=s["top_k"],
                                  top_p=s["top_p"], min_p=s["min_p"], probs=s.get("probs"))
        return (tokens, s["probs"]) if c["probs"] else tokens
    if c["op"] == "fork":
        f = zf.fork_requests(s["table"], s["lens"], s["held"], s["src"], s["dst"], s["free"], s["free_pos"], c["page"])
        zf.q4_copy_pages(s["cache"], f.copy_src, f.copy_dst)
        return (s["table"], f.seq_lens, f.pages_held, f.free_pos, f.copy_src, f.copy_dst, s["records"])
    r = zf.release_requests(s["table"], s["lens"], s["held"], s["release"], s["free"], s["free_pos"], s["pool"])
    m = zf.compact_pages(s["table"], r.pages_held, s["pool"])
    zf.q4_copy_pages(s["cache"], m.copy_src, m.copy_dst)
    return (r.seq_lens, r.pages_held, r.free_pos, s["free"], m.page_table, m.free_pages, m.free_pos, m.copy_src, m.copy_dst,
            s["records"])


# ------------------------------------------------------------------------------------ in 64 bits
def _exact_e4m3(byte):
    e, m = (byte.long() >> 3) & 15, (byte.long() & 7).double()
    return torch.where(e > 0, (8 + m) * torch.exp2(e.double() - 10), m * 2.0 ** -9)


def _exact_e2m1(nibble):
    n = nibble.long()
    e, m = (n >> 1) & 3, (n & 1).double()
    mag = torch.where(e > 0, (2 + m) * torch.exp2(e.double() - 2), m * 0.5)
    return torch.where(n > 7, -mag, mag)


def _exact_kv(rec, hkv):
    """Records [hkv, n, 2304] -> keys and values [hkv, 16 n, 128] in 64 bits."""
    dev = rec.device
    tok, blk = torch.arange(TILE, device=dev), torch.arange(D // G, device=dev)
    k_at = 2048 + (tok % 8 * 16 + tok // 8 * 2)[:, None] + (blk // 2 * 4 + blk % 2)[None]
    v_at = 2176 + (tok % 8 // 2 * 4 + tok // 8 * 2 + tok % 2)[:, None] + (blk * 16)[None]
    byte_at = torch.arange(D // 2, device=dev)[None] ^ (tok // 2 % 2 * 32)[:, None]      # V: halves swapped
    kv = []
    for code_at, scale_at in ((0, k_at), (1024, v_at)):
        byte = rec[..., code_at:code_at + 1024].reshape(hkv, -1, TILE, 64)
        if code_at:
            byte = byte.gather(-1, byte_at.expand(byte.shape))
        x = torch.empty(hkv, byte.shape[1], TILE, D, dtype=torch.float64, device=dev)
        x[..., 0::2] = _exact_e2m1(byte & 15)
        x[..., 1::2] = _exact_e2m1(byte >> 4)
        x *= _exact_e4m3(rec[..., scale_at]).repeat_interleave(G, -1)
        kv.append(x.reshape(hkv, -1, D))
    return kv


def _exact_chunk(case, seed):
    c, s = case, prepare(case, seed)
    hkv, page = c["hkv"], c["page"]
    group = c["hq"] // hkv
    N = s["q"].shape[0]
    out = torch.zeros(N, c["hq"], D, dtype=torch.float64, device="cuda")
    lse = torch.full((N, c["hq"]), -math.inf, dtype=torch.float64, device="cuda")
    row = 0
    for b, (L, T) in enumerate(zip(s["lens"].tolist(), (s["start"][1:] - s["start"][:-1]).tolist())):
        if T == 0:
            continue
        rec = s["records"][s["table"][b, :-(-L // page)].long()].transpose(0, 1).reshape(hkv, -1, RECORD)
        step = max(1, (1 << 27) // (group * L))
        for h in range(hkv):          # a kv head at a time
            k, v = _exact_kv(rec[h:h + 1], 1)
            k, v = k[0, :L], v[0, :L]
            for t0 in range(0, T, step):
                pos = torch.arange(L - T + t0, min(L, L - T + t0 + step), device="cuda")
                last = int(pos[-1]) + 1
                lo = max(0, int(pos[0]) + 1 - c["window"]) if c["window"] else 0
                far = pos[:, None] - torch.arange(lo, last, device="cuda")[None]        # distance back
                q = s["q"][row + t0:row + t0 + len(pos), h * group:(h + 1) * group].double()
                x = torch.einsum("thd,nd->thn", q, k[lo:last]) / math.sqrt(D)
                if c["softcap"]:
                    x = torch.tanh(x / c["softcap"]) * c["softcap"]
                if s["slopes"] is not None:
                    x -= s["slopes"][h * group:(h + 1) * group].double()[None, :, None] * far[:, None]
                dark = (far < 0) if not c["window"] else (far < 0) | (far >= c["window"])
                x = x.masked_fill(dark[:, None], -math.inf)
                z = torch.logsumexp(x, -1)
                lse[row + t0:row + t0 + len(pos), h * group:(h + 1) * group] = z
                out[row + t0:row + t0 + len(pos), h * group:(h + 1) * group] = \
                    torch.einsum("thn,nd->thd", torch.exp(x - z[..., None]), v[lo:last])
        row += T
    return out, lse


def _exact_sample(case, seed):
    s = prepare(case, seed)
    if not case["probs"]:
        return None                   # whole numbers
    rows = []
    for r in range(case["rows"]):     # a row at a time, from the filters' definition
        x = s["logits"][r].double()
        w = torch.softmax(x / s["temperature"][r].double(), 0)
        order = torch.argsort(-x, stable=True)
        n = x.numel()
        if s["top_k"] is not None and int(s["top_k"][r]) > 0:
            n = min(n, int(s["top_k"][r]))
        if s["min_p"] is not None:
            n = min(n, int((w >= s["min_p"][r].double() * w.max()).sum()))
        head = w[order[:n]]
        if s["top_p"] is not None:
            run = torch.cumsum(head, 0) / head.sum()
            n = min(n, int((run < s["top_p"][r].double()).sum()) + 1)
        p = torch.zeros_like(w)
        p[order[:n]] = head[:n] / head[:n].sum()
        rows.append(p)
    return None, torch.stack(rows)


def exact(case, seed):
    if case["op"] == "chunk":
        return _exact_chunk(case, seed)
    if case["op"] == "sample":
        return _exact_sample(case, seed)
    return None                       # whole numbers and copies
