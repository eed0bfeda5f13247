"""Measured cases of the serving and position operators: rotary positions, appending to a paged
key/value cache, attention over that cache (causal or for a tree of drafted tokens), and the
cache's page operations (fork, free, reserve, accept).

Each case names an operator ("op") and its sizes.  `run` makes one pass: the plain forms are
elementary torch operations in 32 bits (64 where 32 lose what matters), rounded once at the end;
with `own` set, the library's calls.  `exact` restates each operator sequence by sequence in 64
bits.  Lengths follow from the case alone, values and page placement from the seed.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BASE = 10000.0


# ------------------------------------------------------------------------------------- cases


def listed():
    return [
        # One decoding step of 64 sequences: q and k are slices of the fused projection's output,
        # one token each at positions far apart.  Launch latency is what counts.
        dict(name="rotary decode", op="rotary", seqs=64, new=1, hq=32, hkv=8, d=128, rot=128,
             dtype="bf16", interleaved=False, backward=False, fused=True, length=32768, factor=4.0),
        # Training on two sequences of 8192 tokens with grouped heads (the GQA workload), forward
        # and backward.
        dict(name="rotary train half", op="rotary", seqs=2, new=8192, hq=32, hkv=8, d=128, rot=128,
             dtype="bf16", interleaved=False, backward=True, fused=False, length=8192, factor=1.0),
        # Training with fp32 activations, interleaved pairs over the first part of a wide head, an
        # odd sequence length.
        dict(name="rotary train part fp32", op="rotary", seqs=4, new=2047, hq=16, hkv=16, d=192,
             rot=64, dtype="fp32", interleaved=True, backward=True, fused=False, length=4096,
             factor=1.0),
        # A decoding step's new keys and values into the cache of one layer, q and k rotated on
        # the way.
        dict(name="append decode", op="append", seqs=64, new_lo=1, new_hi=1, ctx_lo=500,
             ctx_hi=2000, hq=32, hkv=8, d=128, rot=128, interleaved=False, page=64),
        # Prompt chunks of different lengths appended behind what is cached.
        dict(name="append prompts", op="append", seqs=8, new_lo=777, new_hi=2048, ctx_lo=0,
             ctx_hi=1500, hq=32, hkv=8, d=128, rot=64, interleaved=True, page=16),
        # One short sequence, one token: the latency of a single user's decoding step.
        dict(name="attend single", op="attend", seqs=1, new_lo=1, new_hi=1, ctx_lo=501, ctx_hi=501,
             hq=16, hkv=16, d=128, page=16, tree=False),
        # Decoding a full batch with long contexts: the cache is read once, bandwidth is the bound.
        dict(name="attend decode batch", op="attend", seqs=64, new_lo=1, new_hi=1, ctx_lo=4096,
             ctx_hi=8191, hq=32, hkv=8, d=128, page=64, tree=False),
        # Small trees of drafted tokens, every head with its own keys, small heads, small pages.
        dict(name="attend small trees", op="attend", seqs=16, new_lo=5, new_hi=26, ctx_lo=700,
             ctx_hi=2048, hq=16, hkv=16, d=64, page=16, tree=True),
        # Trees of 64 drafted tokens over long contexts: tensor work and bandwidth are near one
        # another.
        dict(name="attend long trees", op="attend", seqs=4, new_lo=64, new_hi=64, ctx_lo=30011,
             ctx_hi=32768, hq=32, hkv=8, d=128, page=128, tree=True),
        # A chunk of 2048 prompt tokens over earlier ones (the chunk workload) in wide heads.
        dict(name="attend prompt chunk", op="attend", seqs=2, new_lo=1500, new_hi=2048, ctx_lo=4000,
             ctx_hi=6144, hq=16, hkv=4, d=256, page=64, tree=False),
        # Eight branches of each of eight sequences: whole pages are shared, the last one copied.
        dict(name="fork branches", op="fork", seqs=8, branches=8, layers=8, hkv=8, d=128, page=64,
             len_lo=400, len_hi=2000),
        # A verified step of 64 sequences over all layers: the step's draft is dropped, made room
        # for again, and a path of it accepted.
        dict(name="accept drafts", op="accept", seqs=64, draft=64, layers=32, hkv=8, d=128, page=64,
             len_lo=100, len_hi=500),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "append", "attend", "attend", "attend", "fork", "accept"])
    hkv = rng.choice([1, 2, 4, 8, 16])
    group = rng.choice([1, 2, 3, 4, 6, 8])
    d = rng.choice([64, 96, 128, 192, 256])
    page = rng.choice([16, 32, 64, 128])
    if op == "rotary":
        new = _spread(rng, 1, 8192)
        seqs = _spread(rng, 1, max(1, min(64, 16384 // new)))
        d = rng.choice([40, 64, 80, 96, 128, 192, 256])
        while new > 1 and seqs * new * hkv * (group + 1) * d > 4e7:
            new = new // 2
        rot = rng.choice([d, d, d // 2 // 2 * 2])
        return dict(op=op, seqs=seqs, new=new, hq=hkv * group, hkv=hkv, d=d, rot=rot,
                    dtype=rng.choice(["bf16", "bf16", "fp32"]), interleaved=rng.random() < 0.5,
                    backward=rng.random() < 0.5, fused=rng.random() < 0.5, length=new + 4096,
                    factor=rng.choice([1.0, 2.5, 8.0]))
    if op == "append":
        new = _spread(rng, 1, 2048)
        ctx = _spread(rng, 1, 4000)
        return dict(op=op, seqs=_spread(rng, 1, max(1, min(64, 16384 // new))),
                    new_lo=max(1, new // 2), new_hi=new, ctx_lo=ctx // 3, ctx_hi=ctx,
                    hq=hkv * group, hkv=hkv, d=d, rot=rng.choice([d, d // 2]),
                    interleaved=rng.random() < 0.5, page=page)
    if op == "attend":
        tree = rng.random() < 0.5
        new = rng.choice([1, _spread(rng, 1, 64), _spread(rng, 1, 1024)])
        new = min(new, 200) if tree else new
        ctx = _spread(rng, 16, 32768)
        seqs = _spread(rng, 1, 64)
        while seqs > 1 and seqs * (ctx + new) * hkv * d * 4 > 1.2e9:
            seqs = seqs // 2
        while new > 1 and 4.0 * seqs * new * (ctx + new) * hkv * group * d > 1.3e11:
            new = new // 2
        return dict(op=op, seqs=seqs, new_lo=max(1, new // 2), new_hi=new, ctx_lo=ctx // 2,
                    ctx_hi=ctx, hq=hkv * group, hkv=hkv, d=d, page=page, tree=tree)
    top = _spread(rng, 20, 1500)
    layers = rng.choice([1, 2, 6, 16])
    if op == "fork":
        return dict(op=op, seqs=_spread(rng, 1, 12), branches=rng.choice([1, 2, 5, 8]),
                    layers=layers, hkv=hkv, d=d, page=page, len_lo=top // 4, len_hi=top)
    return dict(op=op, seqs=_spread(rng, 1, 64), draft=_spread(rng, 4, 128), layers=layers,
                hkv=min(hkv, 8), d=min(d, 128), page=page, len_lo=top // 6, len_hi=top // 2 + 1)


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


def _table(length, rot, factor):
    """Cosines and sines [length, rot / 2, 2] in fp32, from angles in 64 bits; positions are
    divided by `factor` (linear scaling for long contexts)."""
    freq = BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = (torch.arange(length, dtype=torch.float64, device=DEV) / factor)[:, None] * freq
    return torch.stack([a.cos(), a.sin()], -1).float()


def _pool(g, rnd, c, held, spare, layers, slots):
    """A cache whose sequences i hold held[i] tokens in pages placed at random; `spare` more pages
    are free and each table row has room for them."""
    page = c["page"]
    used = [-(-n // page) for n in held]
    pages = sum(used) + spare
    width = max(used + [1]) + spare
    place = rnd.permutation(pages)
    table = np.full((slots, width), -1, np.int32)
    at = 0
    for i, n in enumerate(used):
        table[i, :n] = place[at:at + n]
        at += n
    refs = np.zeros(pages, np.int32)
    refs[place[:at]] = 1
    shape = (layers, pages, c["hkv"], page, c["d"])
    return dict(k=_randn(g, shape), v=_randn(g, shape), table=_ints(table.tolist()),
                lengths=_ints(held + [0] * (slots - len(held))), refs=_ints(refs.tolist()))


def prepare(case, seed):
    c = dict(case)
    g, rnd = _gen(seed), np.random.RandomState(seed % (1 << 31))
    s = dict(case=c)
    if c["op"] == "rotary":
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        t = c["seqs"] * c["new"]
        if c["fused"]:  # slices of one projection's output
            x = _randn(g, (t, c["hq"] + 2 * c["hkv"], c["d"]), dt)
            s["q"], s["k"] = x[:, :c["hq"]], x[:, c["hq"]:c["hq"] + c["hkv"]]
        else:
            s["q"], s["k"] = _randn(g, (t, c["hq"], c["d"]), dt), _randn(g, (t, c["hkv"], c["d"]), dt)
        s["table"] = _table(c["length"], c["rot"], c["factor"])
        # a decoding step rotates to the sequences' own positions, training to 0, 1, ...
        s["positions"] = None
        if c["new"] == 1:
            s["positions"] = torch.randint(0, c["length"], (t,), generator=g, device=DEV,
                                           dtype=torch.int32)
        if c["backward"]:
            s["q"], s["k"] = s["q"].detach().requires_grad_(), s["k"].detach().requires_grad_()
            s["gq"], s["gk"] = _randn(g, s["q"].shape, dt), _randn(g, s["k"].shape, dt)
        return s
    n = c["seqs"]
    slots = rnd.permutation(n)
    if c["op"] in ("append", "attend"):
        new, ctx = _lengths(c["new_lo"], c["new_hi"], n), _lengths(c["ctx_lo"], c["ctx_hi"], n)
        held = [0] * n
        for i in range(n):
            held[slots[i]] = ctx[i] + new[i]
        s.update(_pool(g, rnd, c, held, 3, 1, n))
        s["slots"], s["new"], s["ctx"], s["max_new"] = _ints(slots.tolist()), new, ctx, max(new)
        total = sum(new)
        ends = np.cumsum([0] + new)
        # equal lengths are a dense batch, others a packed one
        s["cu"] = None if min(new) == max(new) else _ints(ends.tolist())
        s["seq"] = torch.repeat_interleave(torch.arange(n, device=DEV), torch.tensor(new, device=DEV))
        s["idx"] = torch.arange(total, device=DEV) - torch.tensor(ends[:-1].tolist(), device=DEV)[s["seq"]]
        if c["op"] == "append":
            x = _randn(g, (total, c["hq"] + 2 * c["hkv"], c["d"]))
            a, b = c["hq"], c["hq"] + c["hkv"]
            s["q"], s["k_new"], s["v_new"] = x[:, :a], x[:, a:b], x[:, b:]
            s["table_rot"] = _table(c["ctx_hi"] + c["new_hi"] + 1, c["rot"], 1.0)
        else:
            s["q"] = _randn(g, (total, c["hq"], c["d"]))
            s["mask"] = _tree_words(rnd, new) if c["tree"] else None
    elif c["op"] == "fork":
        held = _lengths(c["len_lo"], c["len_hi"], n)
        many = n * c["branches"]
        s.update(_pool(g, rnd, c, held, many + 2, c["layers"], n + many))
        s["parents"] = _ints([i % n for i in range(many)])
        s["children"] = _ints((n + rnd.permutation(many)).tolist())
    else:
        held = _lengths(c["len_lo"], c["len_hi"], n)
        room = -(-c["draft"] // c["page"]) + 1
        s.update(_pool(g, rnd, c, held, n * room, c["layers"], n))
        s["slots"] = _ints(slots.tolist())
        s["base"] = _ints([held[i] for i in slots])
        most = min(8, c["draft"])
        path = np.sort(np.stack([rnd.permutation(c["draft"])[:most] for _ in range(n)]), 1)
        s["path"], s["accepted"] = _ints(path.tolist()), _ints(rnd.randint(0, most + 1, n).tolist())
        s["none"], s["zeros"] = _ints([[]] * n).view(n, 0), _ints([0] * n)
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


def _own_rotary(s, c):
    import bwd_tiled_attention_gb300 as fa
    qr, kr = fa.rotary(s["q"], s["k"], s["table"], positions=s["positions"], batch=c["seqs"],
                       interleaved=c["interleaved"])
    if not c["backward"]:
        return {"q": qr, "k": kr}
    dq, dk = torch.autograd.grad((qr, kr), (s["q"], s["k"]), (s["gq"], s["gk"]))
    return {"q": qr, "k": kr, "dq": dq, "dk": dk}


def _own_append(s, c):
    import bwd_tiled_attention_gb300 as fa
    q = fa.cache_append(s["cache"], 0, s["slots"], s["k_new"], s["v_new"], q=s["q"],
                        rotary=s["table_rot"], interleaved=c["interleaved"], cu_seqlens=s["cu"])
    return {"q": q, "k": s["k"], "v": s["v"]}


def _own_attend(s, c):
    import bwd_tiled_attention_gb300 as fa
    o, lse = fa.tree_attention(s["q"], s["cache"], 0, s["slots"], mask=s["mask"],
                               cu_seqlens=s["cu"], max_seqlen=s["max_new"])
    return {"o": o, "lse": lse}


def _own_fork(s, c):
    s["cache"].free(s["children"])
    s["cache"].fork(s["parents"], s["children"])
    return _pool_out(s)


def _own_accept(s, c):
    s["cache"].accept(s["slots"], s["base"], s["none"], s["zeros"])
    s["cache"].reserve(s["slots"], c["draft"])
    s["cache"].accept(s["slots"], s["base"], s["path"], s["accepted"])
    return _pool_out(s)


def _pool_out(s):
    return {n: s[n] for n in ("k", "v", "table", "lengths", "refs")}


def _rotate(x, cos, sin, interleaved):
    """x [T, H, d]; cos, sin [T, 1, rot / 2]: the first rot columns rotated, in 32 bits."""
    half = cos.shape[-1]
    x = x.float()
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, x[..., 2 * half:]], -1)


def _plain_rotary(s, c):
    q, k = s["q"].detach(), s["k"].detach()
    pos = s["positions"]
    if pos is None:
        pos = torch.arange(c["seqs"] * c["new"], device=DEV) % c["new"]
    cos, sin = s["table"][pos.long()].unsqueeze(1).unbind(-1)
    out = {"q": _rotate(q, cos, sin, c["interleaved"]).to(q.dtype),
           "k": _rotate(k, cos, sin, c["interleaved"]).to(k.dtype)}
    if c["backward"]:  # the transpose of a rotation turns back
        out["dq"] = _rotate(s["gq"], cos, -sin, c["interleaved"]).to(q.dtype)
        out["dk"] = _rotate(s["gk"], cos, -sin, c["interleaved"]).to(k.dtype)
    return out


def _counts(s):
    """New tokens of each sequence, int64 [seqs]."""
    if s["cu"] is None:
        return torch.full_like(s["slots"], s["max_new"], dtype=torch.int64)
    return (s["cu"][1:] - s["cu"][:-1]).long()


def _plain_append(s, c):
    slots = s["slots"].long()
    at = (s["lengths"][slots] - _counts(s))[s["seq"]] + s["idx"]  # the tokens' places
    cos, sin = s["table_rot"][at].unsqueeze(1).unbind(-1)
    q = _rotate(s["q"], cos, sin, c["interleaved"]).to(s["q"].dtype)
    k = _rotate(s["k_new"], cos, sin, c["interleaved"]).to(s["q"].dtype)
    page = s["table"][slots[s["seq"]], at // c["page"]].long()
    s["k"][0, page, :, at % c["page"]] = k
    s["v"][0, page, :, at % c["page"]] = s["v_new"]
    return {"q": q, "k": s["k"], "v": s["v"]}


def _plain_attend(s, c):
    slots, n, hkv, d = s["slots"].long(), s["max_new"], c["hkv"], c["d"]
    b, g = slots.shape[0], c["hq"] // c["hkv"]
    length = s["lengths"][slots].long()
    ctx = length - _counts(s)
    width = -(-(c["ctx_hi"] + c["new_hi"]) // c["page"])
    pages = s["table"][slots, :width].long().clamp(min=0)
    k = s["k"][0, pages].transpose(1, 2).reshape(b, hkv, -1, d).float()
    v = s["v"][0, pages].transpose(1, 2).reshape(b, hkv, -1, d).float()
    q = torch.zeros(b, n, c["hq"], d, device=DEV)
    q[s["seq"], s["idx"]] = s["q"].float()
    q = q.view(b, n, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * n, d)
    scores = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    drafted = torch.arange(k.shape[2], device=DEV) - ctx[:, None]  # [b, L]: < 0 in the context
    if s["mask"] is None:
        seen = drafted[:, None] <= torch.arange(n, device=DEV)[:, None]
    else:
        bits = (s["mask"][:, :, None] >> torch.arange(64, device=DEV)) & 1
        rows = torch.zeros(b, n, bits.shape[1] * 64, dtype=torch.bool, device=DEV)
        rows[s["seq"], s["idx"]] = bits.flatten(1).bool()
        at = drafted.clamp(0, rows.shape[2] - 1)[:, None].expand(-1, n, -1)
        seen = (drafted < 0)[:, None] | (rows.gather(2, at) & (drafted < rows.shape[2])[:, None])
    seen = seen & (torch.arange(k.shape[2], device=DEV) < length[:, None])[:, None]
    seen = seen[:, None, None].expand(-1, hkv, g, -1, -1).reshape(b, hkv, g * n, -1)
    scores = scores.masked_fill(~seen, -math.inf)
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - m)
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / total
    lse = (m + total.log()).squeeze(-1).view(b, c["hq"], n)
    o = o.view(b, hkv, g, n, d).permute(0, 3, 1, 2, 4).reshape(b, n, c["hq"], d)
    return {"o": o[s["seq"], s["idx"]].to(s["q"].dtype),
            "lse": lse[s["seq"], :, s["idx"]].t().contiguous()}


def _plain_free(s, slots):
    rows = s["table"][slots]
    s["refs"].index_add_(0, rows.clamp(min=0).flatten(), -(rows >= 0).int().flatten())
    s["table"][slots] = -1
    s["lengths"][slots] = 0


def _free_pages(s):
    """All pages, the free ones first, each kind in order."""
    return torch.sort((s["refs"] != 0).byte(), stable=True).indices


def _plain_fork(s, c):
    parents, children = s["parents"].long(), s["children"].long()
    _plain_free(s, children)
    page, order = c["page"], _free_pages(s)
    length = s["lengths"][parents]
    full, part = (length // page).long(), length % page
    need = (part > 0).long()
    fresh = order[need.cumsum(0) - need]
    rows, col = s["table"][parents], torch.arange(s["table"].shape[1], device=DEV)
    mine = torch.where(col < full[:, None], rows, -1)
    mine = torch.where((col == full[:, None]) & (need > 0)[:, None], fresh[:, None].int(), mine)
    s["table"][children] = mine
    s["lengths"][children] = length
    s["refs"].index_add_(0, mine.clamp(min=0).flatten(), (mine >= 0).int().flatten())
    some = need.nonzero().squeeze(1)
    src, dst = rows[some, full[some]].long(), fresh[some]
    held = (torch.arange(page, device=DEV) < part[some][:, None])[None, :, None, :, None]
    for x in (s["k"], s["v"]):
        x[:, dst] = torch.where(held, x[:, src], x[:, dst])
    return _pool_out(s)


def _plain_reserve(s, c, slots, count):
    page, order, width = c["page"], _free_pages(s), s["table"].shape[1]
    length = s["lengths"][slots].long()
    used = (length + page - 1) // page
    need = (length + count + page - 1) // page - used
    k = torch.arange(-(-count // page) + 1, device=DEV)
    valid = k < need[:, None]
    fresh = order[((need.cumsum(0) - need)[:, None] + k).clamp(max=order.shape[0] - 1)]
    at = slots[:, None] * width + used[:, None] + k
    flat = s["table"].view(-1)
    flat[at] = torch.where(valid, fresh.int(), flat[at])
    s["refs"].index_add_(0, fresh.flatten(), valid.int().flatten())
    s["lengths"][slots] += count


def _plain_take(s, c, slots, base, path, accepted):
    page, width = c["page"], s["table"].shape[1]
    if path.shape[1]:
        j = torch.arange(path.shape[1], device=DEV)
        dst = base[:, None] + j
        src = torch.where(j < accepted[:, None], base[:, None] + path, dst)
        a = s["table"][slots[:, None], src // page].long()
        b = s["table"][slots[:, None], dst // page].long()
        for x in (s["k"], s["v"]):
            x[:, b, :, dst % page] = x[:, a, :, src % page]
    used = (s["lengths"][slots].long() + page - 1) // page
    kept = (base + accepted + page - 1) // page
    col = kept[:, None] + torch.arange(-(-c["draft"] // page) + 1, device=DEV)
    valid, at = col < used[:, None], slots[:, None] * width + col
    flat = s["table"].view(-1)
    s["refs"].index_add_(0, flat[at].clamp(min=0).flatten(), -valid.int().flatten())
    flat[at] = torch.where(valid, -1, flat[at])
    s["lengths"][slots] = (base + accepted).int()


def _plain_accept(s, c):
    slots, base = s["slots"].long(), s["base"].long()
    _plain_take(s, c, slots, base, s["none"].long(), s["zeros"].long())
    _plain_reserve(s, c, slots, c["draft"])
    _plain_take(s, c, slots, base, s["path"].long(), s["accepted"].long())
    return _pool_out(s)


_own = dict(rotary=_own_rotary, append=_own_append, attend=_own_attend, fork=_own_fork,
            accept=_own_accept)
_plain = dict(rotary=_plain_rotary, append=_plain_append, attend=_plain_attend, fork=_plain_fork,
              accept=_plain_accept)


# -------------------------------------------------------------------------------------- work


def work(case):
    c = case
    if c["op"] == "rotary":
        t, heads, e = c["seqs"] * c["new"], c["hq"] + c["hkv"], 2 if c["dtype"] == "bf16" else 4
        times = 2 if c["backward"] else 1
        return {"bytes": times * 2.0 * t * heads * c["d"] * e + min(t, c["length"]) * c["rot"] * 4.0,
                "flops": times * 3.0 * t * heads * c["rot"]}
    n = c["seqs"]
    if c["op"] in ("append", "attend"):
        new, ctx = _lengths(c["new_lo"], c["new_hi"], n), _lengths(c["ctx_lo"], c["ctx_hi"], n)
        t = sum(new)
        if c["op"] == "append":
            return {"bytes": 2.0 * t * (c["hq"] + 2 * c["hkv"]) * c["d"] * 2 + t * c["rot"] * 4.0,
                    "flops": 3.0 * t * (c["hq"] + c["hkv"]) * c["rot"]}
        # a row of a tree sees the context and, here, some of the few drafted tokens
        seen = sum(m * x + m * (m + 1) // 2 for m, x in zip(new, ctx))
        held = sum(m + x for m, x in zip(new, ctx))
        return {"bytes": 4.0 * held * c["hkv"] * c["d"] + 4.0 * t * c["hq"] * c["d"] + 4.0 * t * c["hq"],
                "flops": 4.0 * seen * c["hq"] * c["d"]}
    row = c["layers"] * 2.0 * c["hkv"] * c["d"] * 2
    held = _lengths(c["len_lo"], c["len_hi"], n)
    if c["op"] == "fork":
        copied = c["branches"] * sum(x % c["page"] for x in held)
        return {"bytes": 2 * copied * row + 8.0 * c["branches"] * sum(-(-x // c["page"]) for x in held),
                "flops": 0.0}
    most = min(8, c["draft"])
    return {"bytes": 2 * n * (most / 2.0) * row + 8.0 * n * -(-c["draft"] // c["page"]), "flops": 0.0}


# ------------------------------------------------------------------------------------- exact


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    with torch.no_grad():
        return dict(rotary=_exact_rotary, append=_exact_append, attend=_exact_attend,
                    fork=_exact_fork, accept=_exact_accept)[c["op"]](s, c)


def _turn(x, table, pos, interleaved, back=False):
    """The rotation as a complex product in 64 bits."""
    w = torch.view_as_complex(table.double()[pos.long()])[:, None]
    w = w.conj() if back else w
    half = w.shape[-1]
    y = x.detach().double().clone()
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else \
        (slice(0, half), slice(half, 2 * half))
    z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * w
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_rotary(s, c):
    pos = s["positions"]
    if pos is None:
        pos = torch.cat([torch.arange(c["new"], device=DEV)] * c["seqs"])
    out = {n: _turn(s[n], s["table"], pos, c["interleaved"]) for n in ("q", "k")}
    if c["backward"]:
        out["dq"] = _turn(s["gq"], s["table"], pos, c["interleaved"], True)
        out["dk"] = _turn(s["gk"], s["table"], pos, c["interleaved"], True)
    return out


def _exact_append(s, c):
    q, k, v = [], s["k"].double(), s["v"].double()
    t, slots, table = 0, s["slots"].tolist(), s["table"].tolist()
    for i, n in enumerate(s["new"]):
        pos = s["ctx"][i] + torch.arange(n, device=DEV)
        q.append(_turn(s["q"][t:t + n], s["table_rot"], pos, c["interleaved"]))
        kk = _turn(s["k_new"][t:t + n], s["table_rot"], pos, c["interleaved"])
        first = s["ctx"][i]
        while first < s["ctx"][i] + n:
            row = first % c["page"]
            m = min(c["page"] - row, s["ctx"][i] + n - first)
            a = first - s["ctx"][i]
            page = table[slots[i]][first // c["page"]]
            k[0, page, :, row:row + m] = kk[a:a + m].transpose(0, 1)
            v[0, page, :, row:row + m] = s["v_new"][t + a:t + a + m].double().transpose(0, 1)
            first += m
        t += n
    return {"q": torch.cat(q), "k": k, "v": v}


def _exact_attend(s, c):
    total, group = sum(s["new"]), c["hq"] // c["hkv"]
    o = torch.empty(total, c["hq"], c["d"], dtype=torch.float64, device=DEV)
    lse = torch.empty(c["hq"], total, dtype=torch.float64, device=DEV)
    if 4.0 * sum(m * (m + x) for m, x in zip(s["new"], s["ctx"])) * c["hq"] * c["d"] > 5e12:
        return None
    t, slots = 0, s["slots"].tolist()
    for i, n in enumerate(s["new"]):
        length = s["ctx"][i] + n
        pages = s["table"][slots[i], :-(-length // c["page"])].long()
        hide = torch.zeros(n, length, dtype=torch.bool, device=DEV)
        if s["mask"] is None:
            hide[:, s["ctx"][i]:] = torch.ones(n, n, dtype=torch.bool, device=DEV).triu(1)
        else:
            for j in range(n):
                hide[:, s["ctx"][i] + j] = (s["mask"][t:t + n, j // 64] >> (j % 64)) & 1 == 0
        for h in range(c["hkv"]):
            k = s["k"][0, pages, h].double().reshape(-1, c["d"])[:length]
            v = s["v"][0, pages, h].double().reshape(-1, c["d"])[:length]
            for a in range(h * group, (h + 1) * group):
                x = s["q"][t:t + n, a].double() @ k.t() / math.sqrt(c["d"])
                x[hide] = -math.inf
                lse[a, t:t + n] = torch.logsumexp(x, 1)
                o[t:t + n, a] = torch.softmax(x, 1) @ v
        t += n
    return {"o": o, "lse": lse}


def _host(s):
    return s["table"].tolist(), s["lengths"].tolist(), s["refs"].tolist()


def _said(s, table, lengths, refs):
    return {"k": s["k"], "v": s["v"], "table": _ints(table), "lengths": _ints(lengths),
            "refs": _ints(refs)}


def _exact_fork(s, c):
    table, lengths, refs = _host(s)
    for p, ch in zip(s["parents"].tolist(), s["children"].tolist()):
        n = lengths[p]
        for i in range(-(-n // c["page"])):
            if (i + 1) * c["page"] <= n:
                table[ch][i] = table[p][i]
                refs[table[p][i]] += 1
                continue
            new, rows = refs.index(0), n - i * c["page"]
            refs[new] = 1
            table[ch][i] = new
            s["k"][:, new, :, :rows] = s["k"][:, table[p][i], :, :rows]
            s["v"][:, new, :, :rows] = s["v"][:, table[p][i], :, :rows]
        lengths[ch] = n
    return _said(s, table, lengths, refs)


def _exact_accept(s, c):
    table, lengths, refs = _host(s)
    page, slots = c["page"], s["slots"].tolist()
    for a in slots:
        for i in range(-(-lengths[a] // page), -(-(lengths[a] + c["draft"]) // page)):
            table[a][i] = refs.index(0)
            refs[table[a][i]] = 1
        lengths[a] += c["draft"]
    for a, base, path, n in zip(slots, s["base"].tolist(), s["path"].tolist(), s["accepted"].tolist()):
        for j in range(n):
            x, y = base + path[j], base + j
            for t in (s["k"], s["v"]):
                t[:, table[a][y // page], :, y % page] = t[:, table[a][x // page], :, x % page]
        for i in range(-(-(base + n) // page), -(-lengths[a] // page)):
            refs[table[a][i]] -= 1
            table[a][i] = -1
        lengths[a] = base + n
    return _said(s, table, lengths, refs)
