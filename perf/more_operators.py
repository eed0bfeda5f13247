"""Measured cases of the operators that bound a context: attention with a sliding window and a few
first tokens that stay visible (training and prompts, and over the paged cache), the attention
weight that each cached key has received, and the eviction of the keys that received least.

Each case names an operator ("op") and its sizes.  `run` makes one pass: the plain forms are
elementary torch operations in 32 bits, rounded once at the end; with `own` set, the library's
calls.  `exact` restates each operator sequence by sequence in 64 bits.  Lengths follow from the
case alone, values and page placement from the seed.

Visible keys: position p sees key j <= p when p - j < window, or when j < sinks (window 0: all j <= p).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------------- cases


def listed():
    return [
        # Training on one short sequence: launch latency is what counts.
        dict(name="window short", op="window", seqs=1, len_lo=160, len_hi=160, past_lo=0, past_hi=0,
             hq=2, hkv=2, d=64, window=48, sinks=0, backward=True, det=False),
        # Training on packed documents of uneven lengths (the variable-length workload), a window of
        # 1024 and four first tokens.
        dict(name="window packed train", op="window", seqs=16, len_lo=256, len_hi=8192, past_lo=0,
             past_hi=0, hq=16, hkv=16, d=128, window=1024, sinks=4, backward=True, det=False),
        # Training on one long document (the long workload), grouped heads, a window of 4096.
        dict(name="window long train", op="window", seqs=1, len_lo=32768, len_hi=32768, past_lo=0,
             past_hi=0, hq=16, hkv=4, d=128, window=4096, sinks=16, backward=True, det=False),
        # A prompt's chunks behind earlier tokens, forward only, wide heads.
        dict(name="window prompt chunk", op="window", seqs=2, len_lo=1500, len_hi=2048, past_lo=4000,
             past_hi=6144, hq=16, hkv=4, d=256, window=2000, sinks=64, backward=False, det=False),
        # One token of one user over a long sequence: latency.
        dict(name="cache window single", op="cache", seqs=1, new_lo=1, new_hi=1, ctx_lo=5001,
             ctx_hi=5001, hq=16, hkv=16, d=128, page=16, tree=False, window=512, sinks=4),
        # Decoding a full batch whose contexts are much longer than the window.
        dict(name="cache window decode", op="cache", seqs=64, new_lo=1, new_hi=1, ctx_lo=8192,
             ctx_hi=16383, hq=32, hkv=8, d=128, page=64, tree=False, window=4096, sinks=16),
        # Drafted trees over a window, small heads, small pages.
        dict(name="cache window trees", op="cache", seqs=16, new_lo=5, new_hi=26, ctx_lo=1700,
             ctx_hi=6000, hq=16, hkv=16, d=64, page=16, tree=True, window=1024, sinks=4),
        # What one token of a single user gave to each key: latency.
        dict(name="weights single", op="weights", seqs=1, new_lo=1, new_hi=1, ctx_lo=501, ctx_hi=501,
             hq=16, hkv=16, d=128, page=16),
        # The same behind a decoding step of a full batch: the keys are read once.
        dict(name="weights decode", op="weights", seqs=64, new_lo=1, new_hi=1, ctx_lo=4096,
             ctx_hi=8191, hq=32, hkv=8, d=128, page=64),
        # The last tokens of prompts judge which keys to keep: exponentials are the bound.
        dict(name="weights prompt end", op="weights", seqs=4, new_lo=64, new_hi=128, ctx_lo=8000,
             ctx_hi=16000, hq=32, hkv=8, d=128, page=128),
        # Every few hundred tokens of a batch: the cache goes back to its budget.
        dict(name="evict step", op="evict", seqs=16, keep=2048, recent=512, sinks=4, grow_lo=100,
             grow_hi=256, layers=16, hkv=8, d=128, page=64, prompt=False),
        # Long prompts cut down to a small budget right after they were read.
        dict(name="evict prompts", op="evict", seqs=4, keep=1024, recent=64, sinks=4, grow_lo=7000,
             grow_hi=15000, layers=16, hkv=8, d=128, page=128, prompt=True),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window", "window", "window", "cache", "cache", "weights", "weights", "evict"])
    hkv = rng.choice([1, 2, 4, 8, 16])
    group = rng.choice([1, 2, 3, 4, 8])
    d = rng.choice([64, 96, 128, 192, 256])
    page = rng.choice([16, 32, 64, 128])
    sinks = rng.choice([0, 0, 1, 4, _spread(rng, 1, 300)])
    if op == "window":
        top = _spread(rng, 40, 16384)
        past = rng.choice([0, 0, _spread(rng, 1, 6000)])
        window = _spread(rng, 8, 4096)
        seqs = _spread(rng, 1, 16)
        while seqs > 1 and seqs * top > 65536:
            seqs = seqs // 2
        while hkv * group > 1 and 14.0 * seqs * top * (window + 512) * hkv * group * d > 3e12:
            hkv, group = max(1, hkv // 2), max(1, group // 2)
        return dict(op=op, seqs=seqs, len_lo=rng.choice([top, max(1, top // 5)]), len_hi=top,
                    past_lo=past // 2, past_hi=past, hq=hkv * group, hkv=hkv, d=d, window=window,
                    sinks=sinks, backward=rng.random() < 0.7, det=rng.random() < 0.4)
    if op in ("cache", "weights"):
        tree = op == "cache" and rng.random() < 0.4
        new = rng.choice([1, _spread(rng, 1, 64), _spread(rng, 1, 1024)])
        new = min(new, 150) if tree else new
        ctx = _spread(rng, 16, 32768)
        window = _spread(rng, 8, 8192)
        seqs = _spread(rng, 1, 64)
        while seqs > 1 and seqs * (ctx + new) * hkv * d * 4 > 1.2e9:
            seqs = seqs // 2
        seen = min(ctx, window) if op == "cache" else ctx
        while new > 1 and 4.0 * seqs * new * (seen + new) * hkv * group * d > 1e11:
            new = new // 2
        c = dict(op=op, seqs=seqs, new_lo=max(1, new // 2), new_hi=new, ctx_lo=ctx // 2, ctx_hi=ctx,
                 hq=hkv * group, hkv=hkv, d=d, page=page)
        if op == "cache":
            c.update(tree=tree, window=window, sinks=sinks)
        return c
    keep = _spread(rng, 40, 4096)
    prompt = rng.random() < 0.5
    grow = _spread(rng, 2 * keep, 8 * keep) if prompt else _spread(rng, 1, max(2, keep // 2))
    sinks = min(sinks, keep // 4)
    layers, seqs = rng.choice([1, 2, 6, 16]), _spread(rng, 1, 32)
    while seqs > 1 and 4.0 * layers * seqs * (keep + grow) * hkv * d > 4e9:
        seqs = seqs // 2
    while layers > 1 and 4.0 * layers * seqs * (keep + grow) * hkv * d > 4e9:
        layers = layers // 2
    return dict(op=op, seqs=seqs, keep=keep, recent=rng.choice([0, 1, _spread(rng, 1, keep - sinks)]),
                sinks=sinks, grow_lo=max(1, grow // 2), grow_hi=grow, layers=layers, hkv=hkv, d=d,
                page=page, prompt=prompt)


def _lengths(lo, hi, n):
    """n lengths between lo and hi, uneven, the same for every seed."""
    return [lo + int((hi - lo + 1) * ((i * 0.6180339887 + 0.37) % 1.0)) for i in range(n)]


# ----------------------------------------------------------------------------------- prepare


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _pool(g, rnd, c, held, spare, layers, room):
    """A cache whose sequences i hold held[i] tokens in pages placed at random; `spare` more pages
    are free, and each table row has room for `room` tokens."""
    page = c["page"]
    used = [-(-n // page) for n in held]
    pages = sum(used) + spare
    width = -(-room // page)
    place = rnd.permutation(pages)
    table = np.full((len(held), width), -1, np.int32)
    at = 0
    for i, n in enumerate(used):
        table[i, :n] = place[at:at + n]
        at += n
    refs = np.zeros(pages, np.int32)
    refs[place[:at]] = 1
    shape = (layers, pages, c["hkv"], page, c["d"])
    return dict(k=_randn(g, shape), v=_randn(g, shape), table=_ints(table.tolist()),
                lengths=_ints(held), refs=_ints(refs.tolist()))


BLOCK = 256  # queries that the plain form of the windowed attention takes together


def prepare(case, seed):
    c = dict(case)
    g, rnd = _gen(seed), np.random.RandomState(seed % (1 << 31))
    s = dict(case=c)
    n = c["seqs"]
    if c["op"] == "window":
        lens, past = _lengths(c["len_lo"], c["len_hi"], n), _lengths(c["past_lo"], c["past_hi"], n)
        keys = [a + b for a, b in zip(lens, past)]
        s["lens"], s["keys"] = lens, keys
        s["q"] = _randn(g, (sum(lens), c["hq"], c["d"]))
        s["k"], s["v"] = (_randn(g, (sum(keys), c["hkv"], c["d"])) for _ in range(2))
        if c["backward"]:
            s["dout"] = _randn(g, s["q"].shape)
            for x in ("q", "k", "v"):
                s[x].requires_grad_()
        # equal lengths are a dense batch, others a packed one
        s["dense"] = min(lens) == max(lens) and min(keys) == max(keys)
        ends, ends_k = np.cumsum([0] + lens), np.cumsum([0] + keys)
        s["cu"], s["cu_k"] = _ints(ends.tolist()), _ints(ends_k.tolist())
        # blocks of queries: sequence, first query in it
        blocks = [(i, a) for i in range(n) for a in range(0, lens[i], BLOCK)]
        s["blocks"] = torch.tensor(blocks, device=DEV)
        return s
    slots = rnd.permutation(n)
    s["slots"] = _ints(slots.tolist())
    if c["op"] in ("cache", "weights"):
        new, ctx = _lengths(c["new_lo"], c["new_hi"], n), _lengths(c["ctx_lo"], c["ctx_hi"], n)
        held = [0] * n
        for i in range(n):
            held[slots[i]] = ctx[i] + new[i]
        s.update(_pool(g, rnd, c, held, 3, 1, max(held) + 2 * c["page"]))
        s["new"], s["ctx"], s["max_new"], s["most"] = new, ctx, max(new), max(held)
        total = sum(new)
        ends = np.cumsum([0] + new)
        s["cu"] = None if min(new) == max(new) else _ints(ends.tolist())
        s["seq"] = torch.repeat_interleave(torch.arange(n, device=DEV), torch.tensor(new, device=DEV))
        s["idx"] = torch.arange(total, device=DEV) - torch.tensor(ends[:-1].tolist(), device=DEV)[s["seq"]]
        s["q"] = _randn(g, (total, c["hq"], c["d"]))
        s["mask"] = _tree_words(rnd, new) if c.get("tree") else None
        if c["op"] == "weights":
            # the attention that came before has left its sums, and earlier steps their weights
            s["lse"] = _scores(s, c)[1]
            room = s["table"].shape[1] * c["page"]
            s["weights"] = torch.rand((n, c["hkv"], room), generator=g, device=DEV)
    else:
        grow = _lengths(c["grow_lo"], c["grow_hi"], n)
        # a decoding program keeps its sequences at the budget and appends; a prompt is read whole
        held = [0] * n
        for i in range(n):
            held[slots[i]] = c["keep"] + (grow[i] if c["prompt"] else 0)
        spare = 3 if c["prompt"] else n * (-(-c["grow_hi"] // c["page"]) + 1)
        s.update(_pool(g, rnd, c, held, spare, c["layers"], c["keep"] + c["grow_hi"]))
        room = s["table"].shape[1] * c["page"]
        shape = (c["layers"], n, c["hkv"], room)
        # few keys receive most of the weight
        s["weights"] = torch.rand(shape, generator=g, device=DEV).log().square()
        s["counts"] = _ints([c["keep"] + x for x in grow] if c["prompt"] else grow)
        # what the steps since the last eviction have accumulated
        s["fresh"] = torch.rand(shape if c["prompt"] else shape[:3] + (c["grow_hi"],), generator=g,
                                device=DEV).log().square()
    if own:  # the handle that a program keeps; it does no work of its own
        import bwd_tiled_attention_gb300 as fa
        s["cache"] = fa.PagedCache(s["k"], s["v"], s["table"], s["lengths"], s["refs"])
    return s


def _tree_words(rnd, new):
    """Ancestor bits of random trees: token j's parent is one of the four tokens before it, or
    none.  int64 [tokens, words]; bit j of row i: token i sees the sequence's token j."""
    words = -(-max(new) // 64)
    rows = []
    for n in new:
        seen = []
        for j in range(n):
            p = j - 1 - int(rnd.randint(0, 4))
            seen.append((seen[p] if p >= 0 else 0) | (1 << j))
        rows += seen
    out = np.array([[(r >> (64 * w)) & ((1 << 64) - 1) for w in range(words)] for r in rows], np.uint64)
    return torch.from_numpy(out.view(np.int64)).to(DEV)


# --------------------------------------------------------------------------------------- run


def run(s):
    c = s["case"]
    return (_own if own else _plain)[c["op"]](s, c)


def _own_window(s, c):
    import bwd_tiled_attention_gb300 as fa
    kw = dict(causal=True, window=c["window"], sinks=c["sinks"])
    if s["dense"]:
        kw.update(batch=c["seqs"])
    else:
        kw.update(cu_seqlens=s["cu"], max_seqlen=c["len_hi"])
        if c["past_hi"]:
            kw.update(cu_seqlens_k=s["cu_k"], max_seqlen_k=max(s["keys"]))
    if not c["backward"]:
        o, lse = fa.forward(s["q"], s["k"], s["v"], **kw)
        return {"o": o, "lse": lse}
    o = fa.attention(s["q"], s["k"], s["v"], deterministic=c["det"], **kw)
    dq, dk, dv = torch.autograd.grad(o, (s["q"], s["k"], s["v"]), s["dout"])
    return {"o": o, "dq": dq, "dk": dk, "dv": dv}


def _own_cache(s, c):
    import bwd_tiled_attention_gb300 as fa
    o, lse = fa.tree_attention(s["q"], s["cache"], 0, s["slots"], mask=s["mask"],
                               cu_seqlens=s["cu"], max_seqlen=s["max_new"], window=c["window"],
                               sinks=c["sinks"])
    return {"o": o, "lse": lse}


def _own_weights(s, c):
    import bwd_tiled_attention_gb300 as fa
    fa.cache_weights(s["q"], s["lse"], s["cache"], 0, s["slots"], s["weights"],
                     cu_seqlens=s["cu"], max_seqlen=s["max_new"])
    return {"weights": s["weights"]}


def _own_evict(s, c):
    if c["prompt"]:
        s["cache"].free(s["slots"])
    s["cache"].reserve(s["slots"], s["counts"])
    _accumulated(s, c)
    s["cache"].evict(s["slots"], s["weights"], c["keep"], c["recent"], sinks=c["sinks"])
    return _evicted(s)


def _accumulated(s, c):
    """The weights as the steps before the eviction leave them: the new tokens', or all."""
    if c["prompt"]:
        s["weights"].copy_(s["fresh"])
    else:
        s["weights"][..., c["keep"]:c["keep"] + c["grow_hi"]] = s["fresh"]


def _evicted(s):
    return {n: s[n] for n in ("k", "v", "weights", "table", "lengths", "refs")}


def _plain_window(s, c):
    q, k, v = (s[x].detach() for x in ("q", "k", "v"))
    hkv, g, d, w, sinks = c["hkv"], c["hq"] // c["hkv"], c["d"], c["window"], c["sinks"]
    scale = 1.0 / math.sqrt(d)
    seq, first = s["blocks"].unbind(1)
    cu, cu_k = s["cu"].long(), s["cu_k"].long()
    lq, lk = (cu[1:] - cu[:-1])[seq], (cu_k[1:] - cu_k[:-1])[seq]
    # a block's queries, and the keys that some of them may see: the first ones, then a stretch
    row = first[:, None] + torch.arange(BLOCK, device=DEV)
    row_ok = row < lq[:, None]
    at_q = cu[seq][:, None] + row.clamp(max=(lq - 1)[:, None])
    pos = row + (lk - lq)[:, None]
    start = (pos[:, 0] - w + 1).clamp(min=0)
    few = min(sinks, max(s["keys"]))
    wide = min(w + BLOCK, max(s["keys"]))
    key = torch.cat([torch.arange(few, device=DEV).expand(len(seq), -1),
                     start[:, None] + torch.arange(wide, device=DEV)], 1)
    key_ok = (key < lk[:, None]) & torch.cat(
        [torch.arange(few, device=DEV) < start[:, None],
         torch.ones(len(seq), wide, dtype=torch.bool, device=DEV)], 1)
    at_k = cu_k[seq][:, None] + torch.minimum(key, (lk - 1)[:, None])
    seen = key_ok[:, None] & (key[:, None] <= pos[..., None]) & \
        ((pos[..., None] - key[:, None] < w) | (key[:, None] < sinks))
    seen = seen[:, None, None]                                        # [block, 1, 1, row, key]
    qb = q[at_q].float().view(len(seq), BLOCK, hkv, g, d).permute(0, 2, 3, 1, 4)
    kb, vb = (x[at_k].float().permute(0, 2, 1, 3)[:, :, None] for x in (k, v))
    x = (qb @ kb.transpose(-1, -2)).mul_(scale).masked_fill_(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(m.masked_fill(m == -math.inf, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (m + total.log()).squeeze(-1)
    p = p.div_(total.masked_fill(total == 0, 1.0))
    ob = p @ vb

    def rows(y):  # [block, hkv, g, row, d] -> [tokens, hq, d]
        return y.permute(0, 3, 1, 2, 4).reshape(len(seq), BLOCK, c["hq"], d)[row_ok]
    o = rows(ob).to(q.dtype)
    if not c["backward"]:
        lse = lse.permute(0, 3, 1, 2).reshape(len(seq), BLOCK, c["hq"])[row_ok]
        return {"o": o, "lse": lse.t().contiguous()}
    do = s["dout"][at_q].float() * row_ok[..., None, None]
    do = do.view(len(seq), BLOCK, hkv, g, d).permute(0, 2, 3, 1, 4)
    dv = (p.transpose(-1, -2) @ do).sum(2)
    ds = (do @ vb.transpose(-1, -2)).sub_((do * ob).sum(-1, keepdim=True)).mul_(p)
    dq = rows(ds @ kb) * scale
    dk = (ds.transpose(-1, -2) @ qb).sum(2) * scale

    def keys(y):  # [block, hkv, key, d] summed over the blocks
        y = (y.permute(0, 2, 1, 3) * key_ok[..., None, None]).reshape(-1, hkv, d)
        return torch.zeros(k.shape, device=DEV).index_add_(0, at_k.flatten(), y).to(k.dtype)
    return {"o": o, "dq": dq.to(q.dtype), "dk": keys(dk), "dv": keys(dv)}


def _counts(s):
    """New tokens of each sequence, int64 [seqs]."""
    if s["cu"] is None:
        return torch.full_like(s["slots"], s["max_new"], dtype=torch.int64)
    return (s["cu"][1:] - s["cu"][:-1]).long()


def _scores(s, c):
    """Scores of the new tokens over one layer of the cache, hidden ones -inf, and what belongs to
    them: [b, hkv, g, n, keys], lse [hq, T], keys' places [b, keys], V."""
    slots, n, hkv, d = s["slots"].long(), s["max_new"], c["hkv"], c["d"]
    b, g, page = slots.shape[0], c["hq"] // c["hkv"], c["page"]
    window, sinks = c.get("window") or 1 << 30, c.get("sinks", 0)
    length = s["lengths"][slots].long()
    ctx = length - _counts(s)
    # places that may be seen: the first ones, then a stretch up to the end
    start = (ctx - window + 1).clamp(min=0)
    few = min(sinks, s["most"])
    wide = min(window + n, s["most"])
    key = torch.cat([torch.arange(few, device=DEV).expand(b, -1),
                     start[:, None] + torch.arange(wide, device=DEV)], 1)
    ok = (key < length[:, None]) & torch.cat(
        [torch.arange(few, device=DEV) < start[:, None],
         torch.ones(b, wide, dtype=torch.bool, device=DEV)], 1)
    at = torch.minimum(key, (length - 1)[:, None])
    pages = s["table"][slots[:, None], at // page].long()
    k = s["k"][0][pages, :, at % page].float().transpose(1, 2)
    v = s["v"][0][pages, :, at % page].float().transpose(1, 2)
    q = torch.zeros(b, n, c["hq"], d, device=DEV)
    q[s["seq"], s["idx"]] = s["q"].float()
    q = q.view(b, n, hkv, g, d).permute(0, 2, 3, 1, 4)
    x = (q @ k[:, :, None].transpose(-1, -2)).mul_(1.0 / math.sqrt(d))
    token = torch.arange(n, device=DEV)
    drafted = (key - ctx[:, None])[:, None]                           # [b, 1, keys]: < 0 in the context
    if s["mask"] is None:
        pos = (ctx[:, None] + token)[..., None]
        seen = (drafted <= token[:, None]) & ((pos - key[:, None] < window) | (key[:, None] < sinks))
    else:
        bits = ((s["mask"][:, :, None] >> torch.arange(64, device=DEV)) & 1).flatten(1).bool()
        rows = torch.zeros(b, n, bits.shape[1], dtype=torch.bool, device=DEV)
        rows[s["seq"], s["idx"]] = bits
        # a token's position: as many behind the context as others of its own that it sees
        pos = ctx[:, None] + rows.sum(-1) - rows[:, token, token].long()
        near = (pos[..., None] - key[:, None] < window) | (key[:, None] < sinks)
        of_row = drafted.clamp(0, rows.shape[2] - 1).expand(-1, n, -1)
        seen = torch.where(drafted < 0, near, rows.gather(2, of_row) & (drafted < rows.shape[2]))
    seen = (seen & ok[:, None])[:, None, None]
    x = x.masked_fill_(~seen, -math.inf)
    lse = torch.logsumexp(x, -1).reshape(b, c["hq"], n)[s["seq"], :, s["idx"]].t().contiguous()
    return x, lse, key, ok, v


def _plain_cache(s, c):
    x, lse, _, _, v = _scores(s, c)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(m).exp_()
    o = (p @ v[:, :, None]) / p.sum(-1, keepdim=True)
    b, n = v.shape[0], s["max_new"]
    o = o.permute(0, 3, 1, 2, 4).reshape(b, n, c["hq"], c["d"])
    return {"o": o[s["seq"], s["idx"]].to(s["q"].dtype), "lse": lse}


def _plain_weights(s, c):
    x, _, key, ok, _ = _scores(s, c)
    b, n = key.shape[0], s["max_new"]
    lse = torch.full((b, n, c["hq"]), math.inf, device=DEV)
    lse[s["seq"], s["idx"]] = s["lse"].t()
    lse = lse.view(b, n, c["hkv"], -1).permute(0, 2, 3, 1)[..., None]
    p = x.sub_(lse).exp_().sum((2, 3)) * ok[:, None]
    s["weights"][s["slots"].long(), :, :key.shape[1]] += p
    return {"weights": s["weights"]}


def _plain_free(s, slots):
    rows = s["table"][slots]
    s["refs"].index_add_(0, rows.clamp(min=0).flatten(), -(rows >= 0).int().flatten())
    s["table"][slots] = -1
    s["lengths"][slots] = 0


def _plain_reserve(s, c, slots, counts, most):
    """Pages for counts more tokens of each slot, the lowest free index first."""
    page, width = c["page"], s["table"].shape[1]
    order = torch.sort((s["refs"] != 0).byte(), stable=True).indices
    length = s["lengths"][slots].long()
    used = (length + page - 1) // page
    need = (length + counts + page - 1) // page - used
    k = torch.arange(-(-most // page) + 1, device=DEV)
    valid = k < need[:, None]
    fresh = order[((need.cumsum(0) - need)[:, None] + k).clamp(max=order.shape[0] - 1)].int()
    at = (slots[:, None] * width + used[:, None] + k)[valid]
    s["table"].view(-1)[at] = fresh[valid]
    s["refs"][fresh[valid].long()] = 1
    s["lengths"][slots] += counts.int()


def _plain_evict(s, c):
    slots, page = s["slots"].long(), c["page"]
    if c["prompt"]:
        _plain_free(s, slots)
    _plain_reserve(s, c, slots, s["counts"].long(), c["grow_hi"] + (c["keep"] if c["prompt"] else 0))
    _accumulated(s, c)
    keep, recent, sinks = c["keep"], c["recent"], c["sinks"]
    top, gap = keep - recent - sinks, keep - recent
    length = s["lengths"][slots].long()                               # all above keep
    most = keep + c["grow_hi"]
    w = s["weights"][:, slots, :, :most]                              # [layers, n, hkv, most]
    place = torch.arange(most, device=DEV)
    last = (length - recent)[:, None, None]                           # the recent ones begin here
    middle = (place >= sinks) & (place < last)
    order = torch.sort(w.masked_fill(~middle, -1.0), dim=-1, descending=True, stable=True).indices
    stays = torch.zeros(w.shape, dtype=torch.bool, device=DEV)
    stays.scatter_(-1, order[..., :top], True)
    # kept ones beyond the new end of the middle fill the dropped ones' places, both in order
    holes = (middle & ~stays & (place < gap)).nonzero()
    above = (stays & (place >= gap)).nonzero()
    moves = torch.stack([holes, above], -1)                           # [moves, 4, 2]
    layer, which, head = moves[:, 0, 0], moves[:, 1, 0], moves[:, 2, 0]

    def spots(p, slot):  # page and row of places p
        return s["table"][slot, p // page].long(), p % page
    to, frm = spots(moves[:, 3, 0], slots[which]), spots(moves[:, 3, 1], slots[which])
    for x in (s["k"], s["v"]):
        x[layer, to[0], head, to[1]] = x[layer, frm[0], head, frm[1]]
    s["weights"][layer, slots[which], head, moves[:, 3, 0]] = \
        s["weights"][layer, slots[which], head, moves[:, 3, 1]]
    # the recent ones close up
    i = torch.arange(recent, device=DEV)
    frm = spots(length[:, None] - recent + i, slots[:, None])
    to = spots((gap + i).expand(len(slots), -1), slots[:, None])
    for x in (s["k"], s["v"]):
        x[:, to[0], :, to[1]] = x[:, frm[0], :, frm[1]]
    rows = torch.arange(c["hkv"], device=DEV)
    src = (length[:, None] - recent + i)[None, :, None]
    put = s["weights"][:, slots[:, None, None], rows[:, None], src[0]]
    s["weights"][:, slots, :, gap:keep] = put
    tail = (place >= keep) & (place < length[:, None])
    s["weights"][:, slots, :, :most] = s["weights"][:, slots, :, :most].masked_fill(tail[:, None], 0.0)
    # pages behind the budget are free again
    col = torch.arange(s["table"].shape[1], device=DEV)
    drop = (col >= -(-keep // page)) & (col < ((length + page - 1) // page)[:, None])
    mine = s["table"][slots]
    s["refs"].index_add_(0, mine[drop].long(), torch.full_like(mine[drop], -1))
    s["table"][slots] = mine.masked_fill(drop, -1)
    s["lengths"][slots] = keep
    return _evicted(s)


_own = dict(window=_own_window, cache=_own_cache, weights=_own_weights, evict=_own_evict)
_plain = dict(window=_plain_window, cache=_plain_cache, weights=_plain_weights, evict=_plain_evict)


# -------------------------------------------------------------------------------------- work


def _pairs(first, n, window, sinks):
    """Pairs (position, visible key) of positions first .. first + n - 1."""
    p = np.arange(first, first + n, dtype=np.int64)
    p = p[p >= 0]
    start = np.maximum(p - window + 1, 0)
    return int((p - start + 1 + np.minimum(start, sinks)).sum())


def work(case):
    c, n = case, case["seqs"]
    if c["op"] == "window":
        lens, past = _lengths(c["len_lo"], c["len_hi"], n), _lengths(c["past_lo"], c["past_hi"], n)
        pairs = sum(_pairs(b, a, c["window"], c["sinks"]) for a, b in zip(lens, past))
        tq = sum(lens)
        # keys that nobody sees are not read
        tk = sum(min(a + b, a + c["window"] - 1 + c["sinks"]) for a, b in zip(lens, past))
        q, k = 2.0 * tq * c["hq"] * c["d"], 2.0 * tk * c["hkv"] * c["d"]
        if not c["backward"]:
            return {"bytes": 2 * q + 2 * k + 4.0 * tq * c["hq"], "flops": 4.0 * pairs * c["hq"] * c["d"]}
        # q, k, v, dout in; o, dq, dk, dv out; seven products
        return {"bytes": 4 * q + 4 * k, "flops": 14.0 * pairs * c["hq"] * c["d"]}
    if c["op"] in ("cache", "weights"):
        new, ctx = _lengths(c["new_lo"], c["new_hi"], n), _lengths(c["ctx_lo"], c["ctx_hi"], n)
        t = sum(new)
        window, sinks = c.get("window") or 1 << 30, c.get("sinks", 0)
        # (a row of a tree sees some of the few drafted tokens)
        pairs = sum(_pairs(x, m, window, sinks) for m, x in zip(new, ctx))
        held = sum(min(m + x, m + window - 1 + sinks) for m, x in zip(new, ctx))
        row = 2.0 * held * c["hkv"] * c["d"]
        if c["op"] == "cache":
            return {"bytes": 2 * row + 4.0 * t * c["hq"] * c["d"] + 4.0 * t * c["hq"],
                    "flops": 4.0 * pairs * c["hq"] * c["d"]}
        return {"bytes": row + 8.0 * held * c["hkv"] + 2.0 * t * c["hq"] * c["d"] + 4.0 * t * c["hq"],
                "flops": 2.0 * pairs * c["hq"] * c["d"]}
    # all weights are looked at; the recent rows move, and of the others kept those that lie
    # beyond the new end (with weights in no order)
    heads, size = c["layers"] * c["hkv"], 0.0
    for x in _lengths(c["grow_lo"], c["grow_hi"], n):
        top = c["keep"] - c["recent"] - c["sinks"]
        moved = c["recent"] + x * top / max(1.0, top + x)
        size += 4.0 * (c["keep"] + x) + 2 * moved * (4.0 * c["d"] + 4.0) + 4.0 * x
        size += 8.0 * (c["keep"] + x if c["prompt"] else c["grow_hi"])  # the weights written before
    return {"bytes": heads * size, "flops": 0.0}


# ------------------------------------------------------------------------------------- exact


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    with torch.no_grad():
        return dict(window=_exact_window, cache=_exact_cache, weights=_exact_weights,
                    evict=_exact_evict)[c["op"]](s, c)


def _exact_window(s, c):
    if work(c)["flops"] > 6e12:
        return None
    group, scale, step = c["hq"] // c["hkv"], 1.0 / math.sqrt(c["d"]), 2048
    q, k, v = (s[x].detach() for x in ("q", "k", "v"))
    o = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.full((c["hq"], q.shape[0]), -math.inf, dtype=torch.float64, device=DEV)
    grads = [torch.zeros(x.shape, dtype=torch.float64, device=DEV) for x in (q, k, v)] if c["backward"] else None
    t = u = 0
    for n, m in zip(s["lens"], s["keys"]):
        for a in range(0, n, step):
            z = min(n, a + step)
            pos = torch.arange(a, z, device=DEV)[:, None] + (m - n)
            start = max(0, a + m - n - c["window"] + 1)
            few = min(c["sinks"], start)
            j = torch.cat([torch.arange(few, device=DEV), torch.arange(start, min(m, z + m - n), device=DEV)])
            if len(j) == 0:
                continue
            hide = (j > pos) | ((pos - j >= c["window"]) & (j >= c["sinks"]))
            empty = hide.all(1)
            for h in range(c["hq"]):
                kk, vv, qq = k[u + j, h // group].double(), v[u + j, h // group].double(), q[t + a:t + z, h].double()
                x = (qq @ kk.t()).mul_(scale)
                x[hide] = -math.inf
                lse[h, t + a:t + z] = torch.logsumexp(x, 1)
                p = torch.softmax(x, 1)
                p[empty] = 0
                y = p @ vv
                o[t + a:t + z, h] = y
                if grads:
                    do = s["dout"][t + a:t + z, h].double()
                    ds = p * (do @ vv.t() - (do * y).sum(1, keepdim=True)) * scale
                    grads[0][t + a:t + z, h] = ds @ kk
                    grads[1][u + j, h // group] += ds.t() @ qq
                    grads[2][u + j, h // group] += p.t() @ do
        t, u = t + n, u + m
    if grads:
        return {"o": o, "dq": grads[0], "dk": grads[1], "dv": grads[2]}
    return {"o": o, "lse": lse}


def _slot_rows(s, c, slot, length, h):
    pages = s["table"][slot, :-(-length // c["page"])].long()
    return (s[x][0, pages, h].double().reshape(-1, c["d"])[:length] for x in ("k", "v"))


def _exact_cache(s, c):
    if sum(m * (m + x) for m, x in zip(s["new"], s["ctx"])) * 4.0 * c["hq"] * c["d"] > 5e12:
        return None
    total, group = sum(s["new"]), c["hq"] // c["hkv"]
    o = torch.empty(total, c["hq"], c["d"], dtype=torch.float64, device=DEV)
    lse = torch.empty(c["hq"], total, dtype=torch.float64, device=DEV)
    t, slots = 0, s["slots"].tolist()
    for i, n in enumerate(s["new"]):
        ctx = s["ctx"][i]
        length = ctx + n
        hide = torch.ones(n, length, dtype=torch.bool, device=DEV)
        words = None if s["mask"] is None else s["mask"][t:t + n].tolist()
        for r in range(n):
            others = r
            if words:
                mine = [j for j in range(n) if words[r][j // 64] >> (j % 64) & 1]
                others = len([j for j in mine if j != r])
                hide[r, [ctx + j for j in mine]] = False
            else:
                hide[r, max(ctx, length - n + r - c["window"] + 1):ctx + r + 1] = False
                hide[r, ctx:min(ctx + r + 1, max(ctx, c["sinks"]))] = False
            hide[r, max(0, ctx + others - c["window"] + 1):ctx] = False
            hide[r, :min(ctx, c["sinks"])] = False
        for h in range(c["hkv"]):
            k, v = _slot_rows(s, c, slots[i], length, h)
            for a in range(h * group, (h + 1) * group):
                x = s["q"][t:t + n, a].double() @ k.t() / math.sqrt(c["d"])
                x[hide] = -math.inf
                lse[a, t:t + n] = torch.logsumexp(x, 1)
                o[t:t + n, a] = torch.softmax(x, 1) @ v
        t += n
    return {"o": o, "lse": lse}


def _exact_weights(s, c):
    if sum(m * (m + x) for m, x in zip(s["new"], s["ctx"])) * 2.0 * c["hq"] * c["d"] > 5e12:
        return None
    group = c["hq"] // c["hkv"]
    w = s["weights"].double()
    t, slots = 0, s["slots"].tolist()
    for i, n in enumerate(s["new"]):
        length = s["ctx"][i] + n
        later = torch.ones(n, length, dtype=torch.bool, device=DEV).triu(s["ctx"][i] + 1)
        for h in range(c["hkv"]):
            k, _ = _slot_rows(s, c, slots[i], length, h)
            for a in range(h * group, (h + 1) * group):
                x = s["q"][t:t + n, a].double() @ k.t() / math.sqrt(c["d"]) - s["lse"][a, t:t + n, None].double()
                w[slots[i], h, :length] += x.exp().masked_fill(later, 0.0).sum(0)
        t += n
    return {"weights": w}


def _exact_evict(s, c):
    page, slots = c["page"], s["slots"].tolist()
    if 1.0 * c["layers"] * c["seqs"] * c["hkv"] * (c["keep"] + c["grow_hi"]) > 4e7:
        return None
    table, lengths, refs = (s[x].tolist() for x in ("table", "lengths", "refs"))
    if c["prompt"]:
        for a in slots:
            for i in range(-(-lengths[a] // page)):
                refs[table[a][i]] -= 1
                table[a][i] = -1
            lengths[a] = 0
    for a, n in zip(slots, s["counts"].tolist()):
        for i in range(-(-lengths[a] // page), -(-(lengths[a] + n) // page)):
            table[a][i] = refs.index(0)
            refs[table[a][i]] = 1
        lengths[a] += n
    _accumulated(s, c)
    w = s["weights"].cpu().numpy()
    keep, gap, first = c["keep"], c["keep"] - c["recent"], c["sinks"]
    moved = []
    for a in slots:
        n, pages = lengths[a], np.array(table[a])
        end = n - c["recent"]
        for layer in range(c["layers"]):
            for h in range(c["hkv"]):
                row = w[layer, a, h]
                order = np.argsort(-row[first:end], kind="stable")[:gap - first] + first
                kept = np.zeros(n, bool)
                kept[order] = True
                to = np.concatenate([np.flatnonzero(~kept[first:gap]) + first, np.arange(gap, keep)])
                frm = np.concatenate([np.flatnonzero(kept[gap:end]) + gap, np.arange(end, n)])
                row[to] = row[frm]
                row[keep:n] = 0
                moved.append(np.stack([np.full(len(to), layer), np.full(len(to), h), pages[to // page],
                                       to % page, pages[frm // page], frm % page]))
        for i in range(-(-keep // page), -(-n // page)):
            refs[table[a][i]] -= 1
            table[a][i] = -1
        lengths[a] = keep
    m = torch.from_numpy(np.concatenate(moved, 1)).to(DEV)
    for x in (s["k"], s["v"]):
        x[m[0], m[2], m[1], m[3]] = x[m[0], m[4], m[1], m[5]]
    return {"k": s["k"], "v": s["v"], "weights": torch.from_numpy(w).to(DEV).double(),
            "table": _ints(table), "lengths": _ints(lengths), "refs": _ints(refs)}
