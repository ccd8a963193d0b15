"""Measured cases of the operators of a speculative decode step over a 4-bit paged cache.

write   zf_q4_write_tokens + zf_q4_read_tokens: tokens quantised into pages, and read back as values
attn    zf_q4_decode_attn: decode attention of one or several new tokens over the 4-bit cache
map     zf_map_tokens: block tables and slot maps from request lengths
verify  zf_verify_drafts: accept drafted tokens against the target's probabilities, sample one more

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
def listed():
    return [
        # one request of the tiny configuration: latency of a short call
        dict(name="attn_b1_ctx512", op="attn", batch=1, hq=32, hkv=8, tokens=1, page=16, ctx=512, ctx_min=512),
        # a served batch with ragged contexts (the batched 8B configuration)
        dict(name="attn_b64_ragged", op="attn", batch=64, hq=32, hkv=8, tokens=1, page=16, ctx=8192, ctx_min=1024),
        # the largest batch of the GQA-7 configuration
        dict(name="attn_b128_gqa7", op="attn", batch=128, hq=28, hkv=4, tokens=1, page=16, ctx=8192, ctx_min=8192),
        # the same heads with four new tokens per request: speculative verification, 28 columns per kv head
        dict(name="attn_b32_gqa7_t4", op="attn", batch=32, hq=28, hkv=4, tokens=4, page=16, ctx=8192, ctx_min=8192),
        # the long-context configuration
        dict(name="attn_b4_long", op="attn", batch=4, hq=32, hkv=8, tokens=1, page=64, ctx=131072, ctx_min=131072),
        # a decode step's new tokens of 64 requests
        dict(name="write_b64", op="write", n=64, hkv=8, page=16),
        # an 8192-token prompt
        dict(name="write_prompt", op="write", n=8192, hkv=8, page=16),
        # slots of a speculative step (four drafts and the last token) of 64 requests
        dict(name="map_b64", op="map", batch=64, page=16, ctx=8192, new_min=5, new=5),
        # prompts of 128 requests admitted at once, ragged
        dict(name="map_prompts", op="map", batch=128, page=16, ctx=0, new_min=1, new=8192),
        # one request, four drafts
        dict(name="verify_b1", op="verify", batch=1, drafts=4, vocab=32000, draft_probs=True),
        # a served batch, a large vocabulary
        dict(name="verify_b64", op="verify", batch=64, drafts=4, vocab=128000, draft_probs=True),
        # drafts looked up in the prompt (no draft distribution), odd vocabulary
        dict(name="verify_b128_lookup", op="verify", batch=128, drafts=7, vocab=50001, draft_probs=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "write", "map", "verify"])
    if op == "attn":
        hkv = rng.choice([1, 2, 4, 8, 16, 32])
        group = rng.randint(1, 8)
        tokens = rng.choice([1, 1, 1, 2, 3, 4, 5, 8])
        batch = _log(rng, 1, 128)
        # at most the largest listed case's cache, and its score matrix several times over at most
        ctx = _log(rng, 1, max(2, min(131072, 4194304 // (batch * hkv), 268435456 // (batch * hkv * group * tokens))))
        return dict(op=op, batch=batch, hq=hkv * group, hkv=hkv, tokens=tokens, page=rng.choice([16, 32, 48, 64, 128]),
                    ctx=ctx, ctx_min=rng.choice([ctx, max(1, ctx // 8), 0]))
    if op == "write":
        hkv = rng.choice([1, 2, 3, 4, 8, 16, 32])
        return dict(op=op, n=_log(rng, 1, 65536 // hkv), hkv=hkv, page=rng.choice([16, 32, 48, 64, 128]))
    if op == "map":
        batch = _log(rng, 1, 1024)
        new = _log(rng, 1, min(8192, 1048576 // batch))
        return dict(op=op, batch=batch, page=rng.choice([16, 32, 48, 64, 128]), ctx=rng.choice([0, _log(rng, 1, 8192)]),
                    new_min=rng.choice([0, 1, new]), new=new)
    batch = _log(rng, 1, 128)
    return dict(op=op, batch=batch, drafts=rng.randint(1, 8), vocab=_log(rng, 1000, 8192000 // batch if batch > 64 else 128000),
                draft_probs=rng.random() < 0.6)


def work(case):
    c = case
    if c["op"] == "attn":
        total = c["batch"] * (c["ctx"] + c["ctx_min"]) / 2
        rows = c["batch"] * c["tokens"] * c["hq"]
        pages = total / c["page"] + c["batch"] / 2
        return {"bytes": total * c["hkv"] * RECORD / TILE + rows * (2 * D + 4 * D + 4) + 4 * pages + 4 * c["batch"],
                "flops": 4.0 * D * total * c["hq"] * c["tokens"]}
    if c["op"] == "write":      # source read, records written; records read back, values written
        rows = c["n"] * c["hkv"]
        return {"bytes": rows * (4 * D + 144 + 144 + 4 * D) + 16.0 * c["n"], "flops": 8.0 * rows * D}
    if c["op"] == "map":
        new = c["batch"] * (c["new_min"] + c["new"]) / 2
        return {"bytes": 12.0 * new + 4.0 * new / c["page"] * 2 + 28.0 * c["batch"], "flops": 0.0}
    rows = c["batch"] * (1.7 if c["draft_probs"] else 1.0)    # both distributions where a draft was refused
    return {"bytes": 4.0 * rows * c["vocab"] + 24.0 * c["batch"] * (c["drafts"] + 1), "flops": 4.0 * rows * c["vocab"]}


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


def prepare(case, seed):
    c, g = case, _gen(seed)
    state = dict(case=c)
    if c["op"] == "attn":
        B, page = c["batch"], c["page"]
        lens = torch.randint(c["ctx_min"], c["ctx"] + 1, (B,), generator=g, device="cuda")
        max_pages = -(-c["ctx"] // page)
        pool = int(((lens + page - 1) // page).sum()) + 1
        table, _, _ = _pages_of(lens, page, max_pages, pool, g)
        # records drawn from a pool of quantised token groups
        tiles = pool * c["hkv"] * (page // TILE)
        k, v = _kv(2048 * TILE, 1, g)
        bank = _records(k.view(2048, TILE, D), v.view(2048, TILE, D))
        pick = torch.randint(0, 2048, (tiles,), generator=g, device="cuda")
        records = bank[pick].view(pool, c["hkv"], page // TILE, RECORD)
        q = torch.randn(B, c["tokens"], c["hq"], D, generator=g, device="cuda").to(torch.bfloat16)
        state.update(records=records, table=table, lens=lens.to(torch.int32), q=q)
    elif c["op"] == "write":
        n, page = c["n"], c["page"]
        k, v = _kv(n, c["hkv"], g)
        pool = -(-n // page) + 3
        perm = torch.randperm(pool, generator=g, device="cuda")
        at = torch.arange(n, device="cuda") + 5           # the first page is already partly filled
        state.update(k=k, v=v, page_ids=perm[at // page].to(torch.int32), positions=(at % page).to(torch.int32),
                     records=torch.zeros(pool, c["hkv"], page // TILE, RECORD, dtype=torch.uint8, device="cuda"),
                     pool=pool)
    elif c["op"] == "map":
        B, page = c["batch"], c["page"]
        lens = torch.randint(0, c["ctx"] + 1, (B,), generator=g, device="cuda")
        new = torch.randint(c["new_min"], c["new"] + 1, (B,), generator=g, device="cuda")
        max_pages = -(-(c["ctx"] + c["new"]) // page) + 1
        # some requests hold a page more than their tokens need (drafts that were refused)
        spare = torch.randint(0, 2, (B,), generator=g, device="cuda") * (c["ctx"] > 0)
        held = (lens + page - 1) // page + spare
        need = int(held.sum()) + int(((lens + new + page - 1) // page).sum())
        table, held, perm = _pages_of(held * page, page, max_pages, need + 1, g)
        state.update(lens=lens.to(torch.int32), new=new.to(torch.int32), held=held.to(torch.int32), table=table,
                     free=perm[int(held.sum()):].contiguous(),
                     free_pos=torch.zeros(1, dtype=torch.int32, device="cuda"), max_tokens=B * c["new"])
    else:
        B, T, V = c["batch"], c["drafts"], c["vocab"]
        logits = 3.0 * torch.randn(B, T + 1, V, generator=g, device="cuda")
        target = torch.softmax(logits, -1)
        draft_probs = None
        if c["draft_probs"]:
            draft_probs = torch.softmax(logits[:, :T] + 0.7 * torch.randn(B, T, V, generator=g, device="cuda"), -1)
            source = draft_probs
        else:
            source = target[:, :T]
        drafts = torch.multinomial(source.reshape(B * T, V), 1, generator=g).view(B, T).to(torch.int32)
        if not c["draft_probs"]:      # a lookup proposes likely tokens: the largest for most places
            likely = target[:, :T].argmax(-1).to(torch.int32)
            drafts = torch.where(torch.rand(B, T, generator=g, device="cuda") < 0.7, likely, drafts)
        n = torch.randint(0, T + 1, (B,), generator=g, device="cuda").to(torch.int32) if B > 1 else \
            torch.full((B,), T, dtype=torch.int32, device="cuda")
        state.update(target=target, draft_probs=draft_probs, drafts=drafts.contiguous(), n=n,
                     uniform=torch.rand(B, T + 1, generator=g, device="cuda"))
    return _handles(state) if own else state


def _handles(state):
    """What a user's program of the library keeps: the cache object and the attention workspace."""
    from decode_attention_compressed_gb300 import zf
    c = state["case"]
    if c["op"] in ("attn", "write"):
        state["cache"] = zf.Q4Cache(state["records"].shape[0], c["hkv"], c["page"], records=state["records"])
    if c["op"] == "attn":
        state["workspace"] = zf.new_workspace(zf.q4_workspace_size(c["batch"], c["tokens"], c["hq"], c["hkv"], c["page"],
                                                                   state["table"].shape[1]))
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
def _plain_attn(s):
    c = s["case"]
    B, T, hkv, page = c["batch"], c["tokens"], c["hkv"], c["page"]
    group = c["hq"] // hkv
    k, v = _unrecord(s["records"][s["table"].clamp(min=0).long()])     # [B, pages, hkv, tiles, 16, 128]
    k = k.transpose(1, 2).reshape(B, hkv, -1, D)
    v = v.transpose(1, 2).reshape(B, hkv, -1, D)
    q = s["q"].float().view(B, T, hkv, group, D).permute(0, 2, 1, 3, 4).reshape(B, hkv, T * group, D)
    x = torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(D))
    last = s["lens"][:, None] - T + torch.arange(T, device=x.device)[None]                # last visible position
    seen = torch.arange(k.shape[2], device=x.device)[None, None] <= last[:, :, None]
    x = x.view(B, hkv, T, group, -1).masked_fill(~seen[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, hkv, T * group, -1), v).view(B, hkv, T, group, D) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (torch.log(total) + top)[..., 0]
    return o.permute(0, 2, 1, 3, 4).reshape(B, T, c["hq"], D), lse.permute(0, 2, 1, 3).reshape(B, T, c["hq"])


def _plain_write(s):
    c = s["case"]
    page, slots = s["page_ids"].long(), s["positions"].long()
    out = []
    for x in (s["k"], s["v"]):
        codes, scales = _quantise(x)
        pages = torch.zeros(s["pool"], c["page"], c["hkv"], D // 2, dtype=torch.uint8, device=x.device)
        scale_pages = torch.zeros(s["pool"], c["page"], c["hkv"], D // G, dtype=torch.uint8, device=x.device)
        pages[page, slots] = _pack(codes)
        scale_pages[page, slots] = scales.view(torch.uint8)
        out.append(_values(pages[page, slots], scale_pages[page, slots].view(torch.float8_e4m3fn)).to(torch.bfloat16))
    return tuple(out)


def _plain_map(s):
    c = s["case"]
    page, n_max = c["page"], s["max_tokens"]
    lens, new, held, pos = s["lens"].long(), s["new"].long(), s["held"].long(), s["free_pos"].long()
    need = (lens + new + page - 1) // page
    extra = (need - held).clamp(min=0)
    fits = (extra.sum() + pos <= s["free"].shape[0]) & (new.sum() <= n_max)
    new, extra = new * fits, extra * fits
    base = torch.cumsum(extra, 0) - extra + pos
    j = torch.arange(s["table"].shape[1], device=lens.device)[None]
    fresh = (j >= held[:, None]) & (j < (held + extra)[:, None])
    at = (base[:, None] + j - held[:, None]).clamp(0, s["free"].shape[0] - 1)
    table = torch.where(fresh, s["free"][at], s["table"])
    end = torch.cumsum(new, 0)
    i = torch.arange(n_max, device=lens.device)
    req = torch.searchsorted(end, i, right=True)
    live = req < lens.shape[0]
    req = req.clamp(max=lens.shape[0] - 1)
    at = lens[req] + i - (end - new)[req]
    none = torch.full_like(at, -1)
    page_ids = torch.where(live, table[req, (at // page).clamp(max=table.shape[1] - 1)].long(), none)
    start = torch.cat((torch.zeros(1, dtype=torch.long, device=lens.device), end))
    return tuple(x.to(torch.int32) for x in (table, lens + new, held + extra, pos + extra.sum(), start, page_ids,
                                             torch.where(live, at % page, none), torch.where(live, at, none)))


def _plain_verify(s):
    target, probs, drafts = s["target"], s["draft_probs"], s["drafts"].long()
    B, T = drafts.shape
    n = s["n"].long()
    p = target[:, :T].gather(-1, drafts[..., None])[..., 0]
    q = torch.ones_like(p) if probs is None else probs.gather(-1, drafts[..., None])[..., 0]
    ok = (s["uniform"][:, :T] * q < p) & (torch.arange(T, device=p.device)[None] < n[:, None])
    a = ok.long().cumprod(-1).sum(-1)
    row = torch.arange(B, device=p.device)
    pa = target[row, a]
    at = a.clamp(max=T - 1)
    if probs is None:
        qa = torch.zeros_like(pa).scatter(1, drafts[row, at][:, None], 1.0)
    else:
        qa = probs[row, at]
    w = torch.where((a < n)[:, None], (pa - qa).clamp(min=0), pa)
    w = torch.where((w > 0).any(-1, keepdim=True), w, pa).double()
    cum = torch.cumsum(w, -1)
    token = (cum <= (s["uniform"][:, T].double() * cum[:, -1])[:, None]).sum(-1).clamp(max=w.shape[1] - 1)
    i = torch.arange(T + 1, device=p.device)[None]
    padded = torch.cat((drafts, drafts[:, :1]), 1)
    none = torch.full_like(padded, -1)
    tokens = torch.where(i < a[:, None], padded, torch.where(i == a[:, None], token[:, None], none))
    return a.to(torch.int32), tokens.to(torch.int32)


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"attn": _plain_attn, "write": _plain_write, "map": _plain_map, "verify": _plain_verify}[c["op"]](s)
    from decode_attention_compressed_gb300 import zf
    if c["op"] == "attn":
        return zf.q4_decode_attn(s["cache"], s["q"], s["table"], s["lens"], workspace=s["workspace"])
    if c["op"] == "write":
        zf.q4_write_tokens(s["cache"], s["k"], s["v"], s["page_ids"], s["positions"])
        k, v = zf.q4_read_tokens(s["cache"], s["page_ids"], s["positions"])
        return k.view(torch.bfloat16), v.view(torch.bfloat16)
    if c["op"] == "map":
        m = zf.map_tokens(s["table"], s["lens"], s["held"], s["new"], s["free"], s["free_pos"], c["page"], s["max_tokens"])
        return (s["table"], m.seq_lens, m.pages_held, m.free_pos, m.token_start, m.page_ids, m.positions, m.seq_positions)
    return zf.verify_drafts(s["target"], s["drafts"], s["uniform"], draft_probs=s["draft_probs"], n_drafts=s["n"])


# ------------------------------------------------------------------------------------ in 64 bits
def _exact_e4m3(byte):
    e, m = (byte.long() >> 3) & 15, (byte.long() & 7).double()
    return torch.where(e > 0, (8 + m) * torch.exp2(e.double() - 10), m * 2.0 ** -9)


def _exact_e2m1(nibble):
    n = nibble.long()
    e, m = (n >> 1) & 3, (n & 1).double()
    mag = torch.where(e > 0, (2 + m) * torch.exp2(e.double() - 2), m * 0.5)
    return torch.where(n > 7, -mag, mag)


def _exact_write(x):
    t = x.double().view(*x.shape[:-1], D // G, G)
    a = t.abs().amax(-1)
    want = (a / 6).clamp(min=2.0 ** -9, max=448.0)
    step = torch.exp2(torch.floor(torch.log2(want)).clamp(min=-6) - 3)
    s = (torch.round(want / step) * step)[..., None] * (a > 0)[..., None]
    r = (t.abs() / torch.where(s > 0, s, torch.ones_like(s))).clamp(max=6.0)
    step = torch.where(r < 2, 0.5, torch.where(r < 4, 1.0, 2.0)).double()
    return (torch.sign(t) * torch.round(r / step) * step * s).view(x.shape)


def exact(case, seed):
    c = case
    if c["op"] not in ("attn", "write"):
        return None                 # whole numbers
    s = prepare(case, seed)
    if c["op"] == "write":
        return _exact_write(s["k"]), _exact_write(s["v"])
    B, T, hkv, page = c["batch"], c["tokens"], c["hkv"], c["page"]
    group = c["hq"] // hkv
    out = torch.zeros(B, T, c["hq"], D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, c["hq"]), -math.inf, dtype=torch.float64, device="cuda")
    tok = torch.arange(TILE, device="cuda")
    blk = torch.arange(D // G, device="cuda")
    k_at = 2048 + (tok % 8 * 16 + tok // 8 * 2)[:, None] + (blk // 2 * 4 + blk % 2)[None]
    v_at = 2176 + (tok % 8 // 2 * 4 + tok // 8 * 2 + tok % 2)[:, None] + (blk * 16)[None]
    byte_at = torch.arange(D // 2, device="cuda")[None] ^ (tok // 2 % 2 * 32)[:, None]      # V: halves swapped
    for b in range(B):
        L = int(s["lens"][b])
        if L == 0:
            continue
        rec = s["records"][s["table"][b, :-(-L // page)].long()].transpose(0, 1).reshape(hkv, -1, RECORD)
        kv = []
        for code_at, scale_at in ((0, k_at), (1024, v_at)):
            byte = rec[..., code_at:code_at + 1024].reshape(hkv, -1, TILE, 64)
            if code_at:
                byte = byte.gather(-1, byte_at.expand(byte.shape))
            x = torch.empty(hkv, byte.shape[1], TILE, D, dtype=torch.float64, device="cuda")
            x[..., 0::2] = _exact_e2m1(byte & 15)
            x[..., 1::2] = _exact_e2m1(byte >> 4)
            x *= _exact_e4m3(rec[..., scale_at]).repeat_interleave(G, -1)
            kv.append(x.reshape(hkv, -1, D)[:, :L])
        for t in range(T):
            n = L - T + t + 1
            if n <= 0:
                continue
            q = s["q"][b, t].double().view(hkv, group, D)
            x = torch.einsum("hgd,hnd->hgn", q, kv[0][:, :n]) / math.sqrt(D)
            lse[b, t] = torch.logsumexp(x, -1).reshape(-1)
            out[b, t] = torch.einsum("hgn,hnd->hgd", torch.softmax(x, -1), kv[1][:, :n]).reshape(-1, D)
    return out, lse
