"""Workloads of the scored attention calls and of the cache eviction, with a plain form of each.

Four operators over the NVFP4 paged cache and the FP8 workspace:

  decode   one new token per sequence over the paged cache, its scores capped by a tanh, biased by
           distance, and limited to a window with leading sinks       (nvfp4kv_decode_attention_scored)
  weights  the same, and the softmax weight that every cached token received added to a running sum
           per KV head                                                (nvfp4kv_decode_attention_weights)
  extend   a chunk's queries over the FP8 workspace with the same scores, and with prefix and document
           masks                                                      (nvfp4kv_extend_attention_scored)
  evict    keeping the tokens of largest accumulated weight (and the first and the most recent ones)
           and packing them into fresh pages                          (nvfp4kv_evict)

`run` computes an operator with elementary torch operations in 32 bits, or, with `own` set, by the
library's calls.  `exact` restates the definitions in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE, DIM, PAGE_HEAD = 16, 128, 2304
LOG2E = 1.4426950408889634

# the most that one pass may cost: cached (token, KV head) pairs, and (query, head, key) scores
MOST_CACHED = 4 * 131073 * 8
MOST_SCORES = 64 * 2048 * (16384 + 2048)


def _cached(name, op, batch, low, high, hq, hkv, softcap=0.0, window=0, sinks=0, slopes=False, decay=1.0):
    return {"name": name, "op": op, "batch": batch, "low": low, "high": high, "hq": hq, "hkv": hkv,
            "softcap": softcap, "window": window, "sinks": sinks, "slopes": slopes, "decay": decay}


def _extend(name, batch, prefix, chunk, hq, hkv, softcap=0.0, window=0, sinks=0, slopes=False, full=False, docs=0):
    return {"name": name, "op": "extend", "batch": batch, "prefix": prefix, "chunk": chunk, "hq": hq, "hkv": hkv,
            "softcap": softcap, "window": window, "sinks": sinks, "slopes": slopes, "full": full, "docs": docs}


def _evict(name, batch, low, high, hkv, budget, first, recent):
    return {"name": name, "op": "evict", "batch": batch, "low": low, "high": high, "hkv": hkv, "budget": budget,
            "first": first, "recent": recent}


def listed():
    return [
        # an interactive request or two after a short prompt: the launches' latency is what counts
        _cached("decode_cap_short", "decode", 2, 101, 258, 8, 2, softcap=30.0),
        # a batch of long chats served with a sliding window and a few leading sink tokens
        _cached("decode_window_sinks_8k", "decode", 32, 8193, 8193, 64, 8, window=1024, sinks=4),
        # a continuous batch of very unequal lengths, distance bias
        _cached("decode_bias_ragged", "decode", 96, 512, 32768, 32, 8, slopes=True),
        # long documents answered with capped scores, every cached token visible
        _cached("decode_cap_128k", "decode", 4, 131073, 131073, 64, 8, softcap=50.0),
        # the first decode step after a short prompt, accumulating what each token is worth
        _cached("weights_short", "weights", 1, 777, 777, 8, 1),
        # the decode step of a batch at 8K, every step's weights summed up
        _cached("weights_8k", "weights", 32, 8193, 8193, 64, 8),
        # long contexts with capped scores and a sum that forgets
        _cached("weights_cap_decay_128k", "weights", 4, 100003, 131073, 64, 8, softcap=50.0, decay=0.875),
        # two small prompts whose first half is seen from both sides (an image, an instruction)
        _extend("extend_prefix_mask_short", 2, 100, 33, 8, 2, full=True),
        # documents of some hundred tokens packed into one prompt, capped scores
        _extend("extend_docs_cap_4k", 1, 0, 4099, 32, 8, softcap=30.0, docs=700),
        # the next chunk of a long prompt, capped scores over the whole prefix
        _extend("extend_cap_16k", 1, 16384, 2048, 64, 8, softcap=50.0),
        # a batch at 8K cut down to its 2K most attended tokens
        _evict("evict_8k", 32, 8193, 8193, 8, 2048, 4, 256),
        # long contexts cut down to an eighth
        _evict("evict_128k", 4, 100003, 131073, 8, 16384, 16, 1024),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["decode", "weights", "extend", "evict"])
    hkv = rng.choice([1, 2, 4, 8])
    if op == "extend":
        group = rng.choice([1, 2, 4, 8, 16])
        prefix = rng.choice([0, _log_int(rng, 1, 16384)])
        chunk = _log_int(rng, 1, 4096)
        batch = max(1, min(_log_int(rng, 1, 16), MOST_SCORES // (hkv * group * chunk * (prefix + chunk))))
        while batch * hkv * group * chunk * (prefix + chunk) > MOST_SCORES:
            chunk = max(1, chunk * 3 // 4)
        window = rng.choice([0, 0, _log_int(rng, 1, 8192)])
        return _nameless(_extend("", batch, prefix, chunk, hkv * group, hkv, softcap=rng.choice([0.0, 20.0, 50.0]),
                                 window=window, sinks=rng.choice([0, 4, 37]) if window else 0,
                                 slopes=rng.random() < 0.4, full=rng.random() < 0.3,
                                 docs=rng.choice([0, 0, _log_int(rng, 3, 2000)])))
    high = _log_int(rng, 1 if op != "evict" else 40, 131073)
    low = max(1, high // rng.choice([1, 1, 2, 8, 64]))
    batch = max(1, min(_log_int(rng, 1, 96), MOST_CACHED // (hkv * high)))
    if op == "evict":
        budget = max(16, high // rng.choice([2, 3, 4, 8, 16]))
        first = rng.choice([0, 4, 16, budget // 4])
        return _nameless(_evict("", batch, low, high, hkv, budget, min(first, budget // 2), rng.choice([0, 1, budget // 8, budget // 2])))
    group = rng.choice([1, 2, 4, 5, 8])
    window = rng.choice([0, 0, _log_int(rng, 1, 8192)])
    return _nameless(_cached("", op, batch, low, high, hkv * group, hkv, softcap=rng.choice([0.0, 20.0, 50.0]),
                             window=window, sinks=rng.choice([0, 4, 37]) if window else 0, slopes=rng.random() < 0.4,
                             decay=rng.choice([1.0, 0.875, 0.0]) if op == "weights" else 1.0))


def _nameless(case):
    return {k: v for k, v in case.items() if k != "name"}


def _lengths(case):
    """Cached tokens of each sequence: spread evenly over their logarithm, in mixed order."""
    n, low, high = case["batch"], case["low"], case["high"]
    got = [int(round(low * (high / low) ** (i / (n - 1)))) if n > 1 else high for i in range(n)]
    random.Random(n * 1000003 + high).shuffle(got)
    return got


def _chunks(case):
    """Each sequence's cached prefix and new tokens: the first sequence has the full sizes, later ones less."""
    n = case["batch"]
    share = [1.0 - 0.6 * i / n for i in range(n)]
    return ([int(case["prefix"] * s) for s in share], [max(1, int(case["chunk"] * s)) for s in share])


def _doc_starts(case):
    """For each new token, the sequence position at which its document starts."""
    rng = random.Random(case["docs"] * 7919 + case["chunk"])
    got = []
    for prefix, chunk in zip(*_chunks(case)):
        start, left = 0, rng.randint(1, 2 * case["docs"])
        for pos in range(prefix + chunk):
            if left == 0:
                start, left = pos, rng.randint(1, 2 * case["docs"])
            left -= 1
            if pos >= prefix:
                got.append(start)
    return got


def _full_lens(case):
    """How many leading positions every query of the sequence sees: half of its tokens."""
    return [(p + c) // 2 + 1 for p, c in zip(*_chunks(case))]


def _slopes(heads):
    """Distance-bias slopes: a geometric sequence down to 2^-8."""
    return [2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)]


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _nvfp4_rows(x):
    """E2M1 codes [n, 128] and E4M3 scale bytes [n, 8] of fp32 rows."""
    b = x.view(-1, DIM // 16, 16)
    s = (b.abs().amax(-1) / 6.0).to(torch.float8_e4m3fn)
    y = b / s.float().clamp_min(2.0 ** -9)[..., None]
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    code = torch.bucketize(y.abs(), edges, out_int32=True).to(torch.uint8) | (y < 0).to(torch.uint8) << 3
    return code.view(-1, DIM), s.view(torch.uint8)


def _pool(pages, hkv, gen):
    """A cache pool [pages, hkv, 2304] of keys and values as models make them: channels of unequal size, a few tokens
    that draw attention."""
    pool = torch.empty((pages, hkv, PAGE_HEAD), dtype=torch.uint8, device="cuda")
    channel = torch.exp2(torch.rand(2, DIM, generator=gen, device="cuda") * 3.0 - 1.5)
    for at in range(0, pages, 1 << 15):
        part = pool[at:at + (1 << 15)]
        n = part.shape[0] * hkv * PAGE
        loud = 1.0 + 2.0 * (torch.rand(n, 1, generator=gen, device="cuda") < 0.01)
        k, ks = _nvfp4_rows(torch.randn(n, DIM, generator=gen, device="cuda") * channel[0] * loud)
        v, vs = _nvfp4_rows(torch.randn(n, DIM, generator=gen, device="cuda") * channel[1])
        heads = (part.shape[0], hkv)
        part[..., :1024] = (k[:, 0::2] | k[:, 1::2] << 4).view(*heads, 1024)
        part[..., 1024:1152] = ks.reshape(*heads, 128)
        pairs = v.view(*heads, PAGE // 2, 2, DIM)
        part[..., 1152:2176] = (pairs[..., 0, :] | pairs[..., 1, :] << 4).reshape(*heads, 1024)
        part[..., 2176:] = vs.view(*heads, PAGE, 8).transpose(-1, -2).reshape(*heads, 128)
    return pool


def _page_table(counts, first_page, gen):
    """Pages of each sequence: shuffled ids from first_page on, the rows padded with the first id."""
    order = first_page + torch.randperm(sum(counts), generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(counts), max(counts)), first_page, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = order[at:at + n]
        at += n
    return table


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"op": case["op"], "scale": 1.0 / math.sqrt(DIM)}
    if case["op"] == "evict":
        lens = _lengths(case)
        kept = [min(n, case["budget"]) for n in lens]
        src, dst = [-(-n // PAGE) for n in lens], [-(-n // PAGE) for n in kept]
        s |= {k: case[k] for k in ("budget", "first", "recent", "hkv")}
        s["src_pages"], s["max_len"] = sum(src), max(lens)
        pool = _pool(sum(src), case["hkv"], gen)
        fresh = torch.zeros((sum(dst), case["hkv"], PAGE_HEAD), dtype=torch.uint8, device="cuda")
        s["pool"] = torch.cat((pool, fresh))
        s["table"], s["dst_table"] = _page_table(src, 0, gen), _page_table(dst, sum(src), gen)
        s["lens"] = _int32(lens)
        # accumulated weights: heavy-tailed, with many tokens that never got any
        shape = (case["batch"], case["hkv"], max(lens))
        w = torch.exp(torch.randn(shape, generator=gen, device="cuda") * 2.5 - 4.0)
        s["weights"] = torch.where(torch.rand(shape, generator=gen, device="cuda") < 0.05, torch.zeros_like(w), w)
        s["kept"] = torch.empty((case["batch"], case["hkv"], case["budget"]), dtype=torch.int32, device="cuda")
        s["kept_weights"] = torch.empty((case["batch"], case["hkv"], case["budget"]), device="cuda")
        s["new_lens"] = torch.empty(case["batch"], dtype=torch.int32, device="cuda")
        return s
    hq, hkv = case["hq"], case["hkv"]
    s |= {k: case[k] for k in ("hq", "hkv", "softcap", "window", "sinks")}
    s["slopes"] = torch.tensor(_slopes(hq), dtype=torch.float32, device="cuda") if case["slopes"] else None
    if case["op"] == "extend":
        prefix, chunk = _chunks(case)
        gap = 3  # unused workspace rows behind each sequence
        rows = [p + c + gap for p, c in zip(prefix, chunk)]
        total_rows, total_q = sum(rows), sum(chunk)
        s["max_q_len"], s["max_keys"] = max(chunk), max(p + c for p, c in zip(prefix, chunk))
        s["cu_q"] = torch.tensor(np.concatenate([[0], np.cumsum(chunk)]), dtype=torch.int64, device="cuda")
        s["cu_prefix"] = torch.tensor(np.concatenate([[0], np.cumsum(rows)])[:-1].copy(), dtype=torch.int64, device="cuda")
        s["prefix_lens"] = _int32(prefix)
        s["full_lens"] = _int32(_full_lens(case)) if case["full"] else None
        s["doc_starts"] = _int32(_doc_starts(case)) if case["docs"] else None
        channel = torch.exp2(torch.rand(2, DIM, generator=gen, device="cuda") * 3.0 - 1.5)
        loud = 1.0 + 2.0 * (torch.rand(total_rows, 1, 1, generator=gen, device="cuda") < 0.01)
        draws = torch.randn(2, total_rows, hkv, DIM, generator=gen, device="cuda")
        s["ws_k"] = (draws[0] * channel[0] * loud).to(torch.float8_e4m3fn).view(torch.uint8)
        s["ws_v"] = (draws[1] * channel[1]).to(torch.float8_e4m3fn).view(torch.uint8)
        s["q"] = torch.randn(total_q, hq, DIM, generator=gen, device="cuda").to(torch.bfloat16)
        s["out"] = torch.empty((total_q, hq, DIM), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((total_q, hq), device="cuda")
        return s
    lens = _lengths(case)
    pages = [-(-n // PAGE) for n in lens]
    s["max_len"] = max(lens)
    s["pool"] = _pool(sum(pages), hkv, gen)
    s["table"] = _page_table(pages, 0, gen)
    s["lens"] = _int32(lens)
    s["q"] = torch.randn(case["batch"], hq, DIM, generator=gen, device="cuda").to(torch.bfloat16)
    s["out"] = torch.empty((case["batch"], hq, DIM), dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.empty((case["batch"], hq), device="cuda")
    if case["op"] == "weights":
        s["decay"] = case["decay"]
        s["weights"] = torch.rand((case["batch"], hkv, max(lens)), generator=gen, device="cuda")
    return s


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------

def _e2m1(codes):
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                         device=codes.device)
    return table[codes.to(torch.int32)]


def _dequantised(pool, table):
    """Keys and values [B, Hkv, max_pages * 16, 128] of every page of the tables, in 32 bits."""
    heads = pool[table.long()].transpose(1, 2)                      # [B, Hkv, pages, 2304]
    lead = heads.shape[:3]
    kd = heads[..., :1024].reshape(*lead, PAGE, DIM // 2)
    k = _e2m1(torch.stack((kd & 15, kd >> 4), -1)).view(*lead, PAGE, 8, 16)
    k = k * heads[..., 1024:1152].contiguous().view(torch.float8_e4m3fn).float().view(*lead, PAGE, 8, 1)
    vd = heads[..., 1152:2176].reshape(*lead, PAGE // 2, DIM)
    v = _e2m1(torch.stack((vd & 15, vd >> 4), -2)).view(*lead, PAGE, 8, 16)
    vs = heads[..., 2176:].contiguous().view(torch.float8_e4m3fn).float().view(*lead, 8, PAGE)
    v = v * vs.transpose(-1, -2)[..., None]
    return k.view(*lead[:2], -1, DIM), v.view(*lead[:2], -1, DIM)


def _softmax(scores, visible):
    """Weights and log-sum-exp over the last axis; a row with nothing visible gets zeros and -inf."""
    scores = scores.masked_fill(~visible, -math.inf)
    top = scores.amax(-1, keepdim=True)
    e = (scores - torch.where(torch.isinf(top), torch.zeros_like(top), top)).exp()
    total = e.sum(-1, keepdim=True)
    lse = (torch.where(torch.isinf(top), torch.zeros_like(top), top) + total.log()).squeeze(-1)
    return e / torch.where(total > 0, total, torch.ones_like(total)), lse


def _plain_decode(s):
    b, hkv, group = s["q"].shape[0], s["hkv"], s["hq"] // s["hkv"]
    k, v = _dequantised(s["pool"], s["table"])
    k, v = k[:, :, :s["max_len"]], v[:, :, :s["max_len"]]
    q = s["q"].float().view(b, hkv, group, DIM)
    x = torch.matmul(q, k.transpose(-1, -2)) * s["scale"]            # [B, Hkv, G, L]
    if s["softcap"] > 0:
        x = s["softcap"] * torch.tanh(x / s["softcap"])
    at = torch.arange(s["max_len"], device="cuda")
    lens = s["lens"].long()[:, None]
    if s["slopes"] is not None:
        x = x - s["slopes"].view(1, hkv, group, 1) * (lens - 1 - at).abs().float()[:, None, None]
    visible = at < lens
    if s["window"] > 0:
        visible = visible & ((lens - 1 - at < s["window"]) | (at < s["sinks"]))
    p, lse = _softmax(x, visible[:, None, None])
    out = torch.matmul(p, v).view(b, s["hq"], DIM).to(torch.bfloat16)
    return p, out, lse.view(b, s["hq"])


def _plain_extend(s):
    hkv, group = s["hkv"], s["hq"] // s["hkv"]
    prefix = s["prefix_lens"].long()[:, None]                        # [B, 1]
    chunk = (s["cu_q"][1:] - s["cu_q"][:-1])[:, None]
    at = torch.arange(s["max_keys"], device="cuda")                  # keys
    new = torch.arange(s["max_q_len"], device="cuda")                # queries
    live = new < chunk                                               # [B, C]
    rows = torch.where(at < prefix + chunk, s["cu_prefix"][:, None] + at, torch.zeros_like(at))
    k = s["ws_k"].view(torch.float8_e4m3fn)[rows].float().permute(0, 2, 3, 1)   # [B, Hkv, 128, K]
    v = s["ws_v"].view(torch.float8_e4m3fn)[rows].float().transpose(1, 2)       # [B, Hkv, K, 128]
    mine = torch.where(live, s["cu_q"][:-1, None] + new, torch.zeros_like(new))
    q = s["q"][mine].float().view(*live.shape, hkv, group, DIM).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q, k[:, :, None]) * s["scale"]                  # [B, Hkv, G, C, K]
    if s["softcap"] > 0:
        x = s["softcap"] * torch.tanh(x / s["softcap"])
    pos = (prefix + new)[..., None]                                  # [B, C, 1]
    if s["slopes"] is not None:
        x = x - s["slopes"].view(1, hkv, group, 1, 1) * (pos - at).abs().float()[:, None, None]
    high = pos if s["full_lens"] is None else torch.maximum(pos, s["full_lens"].long()[:, None, None] - 1)
    low = torch.zeros_like(pos) if s["doc_starts"] is None else s["doc_starts"].long()[mine][..., None]
    visible = (at >= low) & (at <= high) & (at < (prefix + chunk)[..., None]) & live[..., None]
    if s["window"] > 0:
        visible = visible & ((pos - at < s["window"]) | (at < low + s["sinks"]))
    p, lse = _softmax(x, visible[:, None, None])
    out = torch.matmul(p, v[:, :, None])                             # [B, Hkv, G, C, 128]
    out = out.permute(0, 3, 1, 2, 4).reshape(*live.shape, s["hq"], DIM)[live].to(torch.bfloat16)
    return {"out": out, "lse": lse.permute(0, 3, 1, 2).reshape(*live.shape, s["hq"])[live]}


def _plain_evict(s):
    b, hkv = s["lens"].shape[0], s["hkv"]
    at = torch.arange(s["max_len"], device="cuda")
    lens = s["lens"].long()[:, None, None]                           # [B, 1, 1]
    count = lens.clamp_max(s["budget"])
    always = (at < s["first"]) | (at >= lens - s["recent"])
    rank = torch.where(always, math.inf, s["weights"])
    rank = torch.where(at < lens, rank, -math.inf)
    n = min(s["budget"], s["max_len"])
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :n]
    slot = torch.arange(n, device="cuda")
    order = torch.where(slot < count, order, s["max_len"])           # [B, Hkv, n]
    order = torch.sort(order, dim=-1).values
    used = slot < count
    s["kept"].fill_(-1)
    s["kept"][..., :n] = torch.where(used, order, -1).to(torch.int32)
    order = torch.where(used, order, 0)
    s["kept_weights"].zero_()
    s["kept_weights"][..., :n] = torch.where(used, s["weights"].gather(-1, order), 0.0)
    s["new_lens"].copy_(count.view(-1))
    # the kept rows' bytes, then the rows of the last pages behind them as zeros
    slots = s["dst_table"].shape[1] * PAGE
    order = torch.cat((order, order.new_zeros(b, hkv, max(0, slots - n))), -1)[..., :slots]
    used = torch.arange(slots, device="cuda") < count
    page = s["table"].long().gather(1, (order // PAGE).view(b, -1)).view(b, hkv, slots)
    row, head = order % PAGE, torch.arange(hkv, device="cuda")[None, :, None]
    keep = used.to(torch.uint8).expand(b, hkv, slots)[..., None]
    pages = s["pool"]
    kd = pages[..., :1024].unflatten(-1, (PAGE, 64))[page, head, row] * keep
    ks = pages[..., 1024:1152].unflatten(-1, (PAGE, 8))[page, head, row] * keep
    vd = pages[..., 1152:2176].unflatten(-1, (PAGE // 2, DIM))[page, head, row // 2]
    vd = (vd >> (4 * (row % 2)).to(torch.uint8)[..., None] & 15) * keep
    vs = pages[..., 2176:].unflatten(-1, (8, PAGE)).transpose(-1, -2)[page, head, row] * keep
    lead = (b, hkv, slots // PAGE)
    pair = vd.view(*lead, PAGE // 2, 2, DIM)
    made = torch.cat((kd.reshape(*lead, 1024), ks.reshape(*lead, 128),
                      (pair[..., 0, :] | pair[..., 1, :] << 4).view(*lead, 1024),
                      vs.reshape(*lead, PAGE, 8).transpose(-1, -2).reshape(*lead, 128)), -1)
    live = torch.arange(slots // PAGE, device="cuda") * PAGE < count[:, 0]       # [B, pages]
    pages[s["dst_table"].long()[live]] = made.transpose(1, 2)[live]
    return _evicted(s)


def _evicted(s):
    # the rows move as they are, so the packed bytes themselves are what comes back
    return {"pages": s["pool"][s["src_pages"]:], "kept": s["kept"], "weights": s["kept_weights"], "lens": s["new_lens"]}


def _plain(s):
    if s["op"] == "evict":
        return _plain_evict(s)
    if s["op"] == "extend":
        return _plain_extend(s)
    p, out, lse = _plain_decode(s)
    if s["op"] == "decode":
        return {"out": out, "lse": lse}
    w = s["weights"]
    at = torch.arange(w.shape[-1], device="cuda")
    now = p.view(p.shape[0], s["hkv"], -1, p.shape[-1]).sum(2)
    w.copy_(torch.where(at < s["lens"][:, None, None], s["decay"] * w + now, w))
    return {"out": out, "lse": lse, "weights": w}


# --------------------------------------------------------------------------
# the library's calls
# --------------------------------------------------------------------------

def _own(s):
    import nvfp4_quantized_paged_quantize_gb300 as kv

    if s["op"] == "evict":
        cache = kv.Cache(s["pool"], s["pool"].shape[0], s["hkv"])
        kv.nvfp4kv_evict(cache, s["table"], s["lens"], s["weights"], s["budget"], s["first"], s["recent"],
                         s["dst_table"], s["kept"], s["kept_weights"], s["new_lens"])
        return _evicted(s)
    scoring = kv.Scoring(softcap=s["softcap"], window=s["window"], sinks=s["sinks"], slopes=s["slopes"])
    if s["op"] == "extend":
        kv.nvfp4kv_extend_attention_scored(s["q"], s["cu_q"], s["max_q_len"], s["ws_k"], s["ws_v"], s["cu_prefix"],
                                           s["prefix_lens"], s["out"], s["scale"], scoring=scoring,
                                           full_lens=s["full_lens"], doc_starts=s["doc_starts"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    b, pages = s["q"].shape[0], s["pool"].shape[0]
    cache = kv.Cache(s["pool"], pages, s["hkv"])
    if s["op"] == "decode":
        if "workspace" not in s:  # scratch of the batch's shape, as a program keeps it between steps
            s["workspace"] = torch.empty(kv.nvfp4kv_decode_workspace_size(cache, b, s["hq"]), dtype=torch.uint8, device="cuda")
        kv.nvfp4kv_decode_attention_scored(cache, s["q"], s["out"], s["table"], s["lens"], s["scale"], s["workspace"],
                                           scoring=scoring, lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if "workspace" not in s:
        n = kv.nvfp4kv_decode_weights_workspace_size(cache, b, s["hq"], pages)
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    kv.nvfp4kv_decode_attention_weights(cache, s["q"], s["out"], s["table"], s["lens"], s["scale"], s["weights"],
                                        s["workspace"], scoring=scoring, decay=s["decay"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"], "weights": s["weights"]}


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def _visible_pages(n, window, sinks):
    """Pages of a sequence of n cached tokens that hold a visible one."""
    pages = -(-n // PAGE)
    if window <= 0 or n <= window:
        return pages
    first = (n - window) // PAGE
    return pages - first + min(first, -(-sinks // PAGE))


def _visible_keys(case):
    """(query, key) pairs of the extend's masks, heads not counted."""
    prefix, chunk = _chunks(case)
    starts = np.array(_doc_starts(case)) if case["docs"] else np.zeros(sum(chunk), dtype=np.int64)
    total, at = 0, 0
    for b, (p, c) in enumerate(zip(prefix, chunk)):
        pos = p + np.arange(c)
        low = starts[at:at + c]
        at += c
        high = np.maximum(pos, min(p + c, _full_lens(case)[b]) - 1) if case["full"] else pos
        near = np.maximum(low, pos - case["window"] + 1) if case["window"] > 0 else low
        sink = np.clip(np.minimum(low + case["sinks"], high + 1) - low, 0, np.maximum(near - low, 0)) if case["window"] > 0 else 0
        total += int(np.sum(np.maximum(high + 1 - near, 0) + sink))
    return total


def work(case):
    if case["op"] == "evict":
        lens = _lengths(case)
        kept = sum(min(n, case["budget"]) for n in lens)
        return {"bytes": case["hkv"] * (4.0 * sum(lens) + kept * (2 * 144 + 8)), "flops": 0}
    hq, hkv = case["hq"], case["hkv"]
    if case["op"] == "extend":
        prefix, chunk = _chunks(case)
        rows, queries = sum(prefix) + sum(chunk), sum(chunk)
        return {"bytes": rows * hkv * 2.0 * DIM + queries * hq * (4 * DIM + 4), "flops": 4.0 * DIM * hq * _visible_keys(case)}
    lens = _lengths(case)
    pages = sum(_visible_pages(n, case["window"], case["sinks"]) for n in lens)
    need = pages * hkv * float(PAGE_HEAD) + len(lens) * hq * (4 * DIM + 4)
    if case["op"] == "weights":
        need += hkv * sum(lens) * (8.0 if case["decay"] else 4.0)
    return {"bytes": need, "flops": 4.0 * DIM * hq * PAGE * pages}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

_E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def _byte_values():
    """The 16 E2M1 codes and the 256 E4M3 bytes as 64-bit numbers, from the formats' fields."""
    e2m1 = np.concatenate([_E2M1, -_E2M1])
    byte = np.arange(256)
    exponent, mantissa = byte >> 3 & 15, byte & 7
    e4m3 = np.where(exponent > 0, (1 + mantissa / 8.0) * 2.0 ** (exponent - 7.0), mantissa / 8.0 * 2.0 ** -6)
    e4m3 = np.where(byte & 128, -e4m3, e4m3)
    return torch.tensor(e2m1, device="cuda"), torch.tensor(e4m3, device="cuda")


def _exact_rows(pool, ids, head, n):
    """Keys and values [n, 128] of one sequence and KV head in 64 bits, row by row of the page layout."""
    e2m1, e4m3 = _byte_values()
    t = torch.arange(n, device="cuda")
    raw = pool[ids.long()[t // PAGE], head]                          # [n, 2304]: each token's page-head
    row, d = (t % PAGE)[:, None], torch.arange(DIM, device="cuda")[None]
    kb = raw.gather(1, row * 64 + d // 2).long()
    kc = torch.where(d % 2 == 0, kb & 15, kb >> 4)
    k = e2m1[kc] * e4m3[raw.gather(1, 1024 + row * 8 + d // 16).long()]
    vb = raw.gather(1, 1152 + row // 2 * 128 + d).long()
    vc = torch.where(row % 2 == 0, vb & 15, vb >> 4)
    v = e2m1[vc] * e4m3[raw.gather(1, 2176 + d // 16 * 16 + row).long()]
    return k, v


def _exact_attend(s, q, k, v, pos, low, high, head):
    """Attention of queries [c, 128] of one head at positions pos over keys [n, 128]; low <= key <= high is visible."""
    x = q.double() @ k.T * s["scale"]
    if s["softcap"] > 0:
        x = s["softcap"] * torch.tanh(x / s["softcap"])
    j = torch.arange(k.shape[0], device="cuda")[None]
    pos, low, high = pos[:, None], low[:, None], high[:, None]
    if s["slopes"] is not None:
        x -= float(s["slopes"][head]) * (pos - j).abs()
    seen = (j >= low) & (j <= high)
    if s["window"] > 0:
        seen &= (j > pos - s["window"]) | (j < low + s["sinks"])
    x[~seen] = -math.inf
    lse = torch.logsumexp(x, 1)
    p = torch.where(seen, torch.exp(x - lse[:, None]), 0.0)
    return p, p @ v, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "evict":
        return _exact_evict(s)
    hkv, group = s["hkv"], s["hq"] // s["hkv"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    if case["op"] == "extend":
        _, e4m3 = _byte_values()
        at = 0
        for b, (p, c) in enumerate(zip(*_chunks(case))):
            first, n = int(s["cu_prefix"][b]), p + c
            low = s["doc_starts"][at:at + c].long() if case["docs"] else torch.zeros(c, dtype=torch.int64, device="cuda")
            pos = p + torch.arange(c, device="cuda")
            high = pos.clamp_min(min(n, _full_lens(case)[b]) - 1) if case["full"] else pos
            for h in range(s["hq"]):
                k = e4m3[s["ws_k"][first:first + n, h // group].long()]
                v = e4m3[s["ws_v"][first:first + n, h // group].long()]
                _, out[at:at + c, h], lse[at:at + c, h] = _exact_attend(s, s["q"][at:at + c, h], k, v, pos, low, high, h)
            at += c
        return {"out": out, "lse": lse}
    weights = s["weights"].double() if case["op"] == "weights" else None
    zero = torch.zeros(group, dtype=torch.int64, device="cuda")
    for b, n in enumerate(_lengths(case)):
        for h in range(hkv):
            k, v = _exact_rows(s["pool"], s["table"][b], h, n)
            ps = []
            for g in range(group):
                i = h * group + g
                p, out[b, i], lse[b, i] = _exact_attend(s, s["q"][b, i][None], k, v, zero[:1] + n - 1, zero[:1], zero[:1] + n - 1, i)
                ps.append(p[0])
            if weights is not None:
                weights[b, h, :n] = case["decay"] * weights[b, h, :n] + torch.stack(ps).sum(0)
    got = {"out": out, "lse": lse}
    return got if weights is None else {**got, "weights": weights}


def _exact_evict(s):
    """The kept weights; the pages and indices are bytes and whole numbers."""
    w = s["weights"].double().cpu().numpy()
    got = np.zeros(s["kept_weights"].shape)
    for b, n in enumerate(s["lens"].tolist()):
        m = min(n, s["budget"])
        for h in range(s["hkv"]):
            forced = sorted(set(range(min(s["first"], n))) | set(range(max(0, n - s["recent"]), n)))
            if m == n:
                keep = np.arange(n)
            else:
                rest = np.setdiff1d(np.arange(n), forced)
                best = rest[np.argsort(-w[b, h, rest], kind="stable")][:m - len(forced)]
                keep = np.sort(np.concatenate([np.array(forced, dtype=np.int64), best]))
            got[b, h, :m] = w[b, h, keep]
    return {"pages": None, "kept": None, "weights": torch.from_numpy(got), "lens": None}
