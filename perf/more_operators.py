"""The operators of a step around paged attention as a user calls them, and their plain form.

  plan     block tables, slot maps, positions and offsets from the lengths of the requests
  rope     norms of queries and keys per head, and the rotation, which may have several axes
  ropegrad its backward pass: gradients of queries, keys and both weights
  append   the same for serving: normed, rotated keys and the values go to their slots in the cache
  shared   attention of a batch whose sequences share prefixes: a prefix's keys serve all of them
"""
import math
import random

import torch

own = False

ROTARY_BASE = 10000.0
EPS = 1e-6


# ---- cases ---------------------------------------------------------------------------------
# new: new tokens per sequence (lo, hi), ctx: tokens already there (lo, hi; of shared: behind the
# prefix).  Lengths come from the case alone ("lens"), values and the order of pages from the seed.

def _plan(name, batch, new, ctx, page, lens=1):
    return {"name": name, "op": "plan", "batch": batch, "new_lo": new[0], "new_hi": new[1],
            "ctx_lo": ctx[0], "ctx_hi": ctx[1], "page": page, "lens": lens}


def _rope(name, op, tokens, heads, kv_heads, dim, rotary, interleaved=False, axes=1, mixed=False,
          norm=True, w32=False, packed=True, page=64):
    """mixed: the axes take planes in turn instead of in sections; packed: q, k, v are parts of
    the rows of one projection; w32: weights in fp32."""
    return {"name": name, "op": op, "tokens": tokens, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "rotary": rotary, "interleaved": interleaved, "axes": axes, "mixed": mixed,
            "norm": norm, "w32": w32, "packed": packed, "page": page}


def _shared(name, groups, size, prefix, new, ctx, heads, kv_heads, dim, page, lens=1):
    """groups of size (lo, hi) sequences, each group behind one prefix of (lo, hi) tokens."""
    return {"name": name, "op": "shared", "groups": groups, "size_lo": size[0], "size_hi": size[1],
            "prefix_lo": prefix[0], "prefix_hi": prefix[1], "new_lo": new[0], "new_hi": new[1],
            "ctx_lo": ctx[0], "ctx_hi": ctx[1], "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "page": page, "lens": lens}


def listed():
    return [
        # one generation step of 64 sequences: latency
        _plan("plan-step", 64, (1, 1), (64, 4096), 64, lens=31),
        # a step that mixes long and short chunks, empty ones among them, on small pages
        _plan("plan-mixed", 333, (0, 1500), (0, 9000), 16, lens=32),
        # queries and keys of a training step of 4 sequences of 4096 tokens
        _rope("rope-train", "rope", 16384, 32, 8, 128, 128),
        # an image's tokens: three axes, odd number of tokens, half of a small head rotated
        _rope("rope-image", "rope", 1369, 6, 3, 64, 32, axes=3, mixed=True, w32=True, packed=False),
        # the training step's backward pass
        _rope("ropegrad-train", "ropegrad", 16384, 32, 8, 128, 128),
        # a short ragged batch with positions of time, height and width, planes interleaved
        _rope("ropegrad-video", "ropegrad", 2011, 14, 2, 128, 96, interleaved=True, axes=3),
        # the cache write of one generation step of 64 sequences: latency
        _rope("append-step", "append", 64, 32, 8, 128, 128, page=256),
        # the cache write of 8 chunks of 2048 tokens
        _rope("append-prompt", "append", 16384, 32, 8, 128, 128, page=256),
        # four answers to one short question: the smallest call, latency
        _shared("shared-short", 1, (4, 4), (512, 512), (1, 1), (1, 100), 8, 2, 64, 64, lens=41),
        # 64 requests behind one long system prompt, one token each
        _shared("shared-prompt", 1, (64, 64), (32768, 32768), (1, 1), (100, 2000), 32, 8, 128, 256,
                lens=42),
        # several documents, some asked once, odd lengths, 7 query heads a kv head, small pages
        _shared("shared-documents", 5, (1, 40), (1001, 30011), (1, 1), (0, 900), 14, 2, 128, 16,
                lens=43),
        # checking 4 drafted tokens of 16 samples behind a prefix of 100K tokens
        _shared("shared-verify", 1, (16, 16), (100001, 100001), (4, 4), (64, 1024), 32, 8, 128, 64,
                lens=44),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "ropegrad", "append", "shared", "shared"])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 7, 8])
    dim = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128, 256])
    lens = rng.randrange(1 << 30)
    if op == "plan":
        batch = _log_int(rng, 1, 1000)
        hi = _log_int(rng, 1, max(1, 240000 // batch))
        c = _plan("", batch, (rng.choice([0, 1, hi]), hi), (0, _log_int(rng, 1, 9000)), page, lens)
    elif op == "shared":
        groups = rng.randint(1, 6)
        size = _log_int(rng, 1, max(1, 64 // groups))
        new = rng.choice([1, 1, 1, rng.randint(2, 8)])
        prefix = _log_int(rng, 16, 90000 * 32 // (max(32, heads) * groups * new))
        c = _shared("", groups, (rng.randint(1, size), size), (rng.randint(1, prefix), prefix),
                    (min(new, 1), new), (0, _log_int(rng, 1, 2000 // new)), heads, kv_heads, dim,
                    page, lens)
    else:
        c = _rope("", op, _log_int(rng, 1, 16384 * 40 * 128 // ((heads + kv_heads) * dim) // 2), heads,
                  kv_heads, dim, rng.choice([16, dim // 2, dim, dim]), rng.random() < 0.3,
                  rng.choice([1, 1, 2, 3]), rng.random() < 0.5, rng.random() < 0.8, rng.random() < 0.3,
                  rng.random() < 0.7, page)
    del c["name"]
    return c


def _plan_lengths(case):
    r = random.Random(case["lens"])
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    return ctx, [max(1, new[0])] + new[1:]


def _shared_lengths(case):
    """Sequences per group, prefix per group, and per sequence its new tokens and all its keys."""
    r = random.Random(case["lens"])
    size = [r.randint(case["size_lo"], case["size_hi"]) for _ in range(case["groups"])]
    prefix = [r.randint(case["prefix_lo"], case["prefix_hi"]) for _ in range(case["groups"])]
    new, keys = [], []
    for n, p in zip(size, prefix):
        for _ in range(n):
            new.append(r.randint(case["new_lo"], case["new_hi"]))
            keys.append(p + r.randint(case["ctx_lo"], case["ctx_hi"]) + new[-1])
    return size, prefix, new, keys


def _sections(case):
    """Planes per axis: time, height, width as 2 : 3 : 3, or halves."""
    half, axes = case["rotary"] // 2, case["axes"]
    if axes == 1:
        return (half,)
    rest = half // axes if case["mixed"] else half * 3 // (4 if axes == 2 else 8)
    return (half - rest * (axes - 1),) + (rest,) * (axes - 1)


def _plane_axis(case):
    """The axis of each plane: in sections, or the axes in turn while their sections last."""
    s = _sections(case)
    if not case["mixed"]:
        return [a for a, n in enumerate(s) for _ in range(n)]
    return [i % len(s) if i // len(s) < s[i % len(s)] else 0 for i in range(case["rotary"] // 2)]


def work(case):
    op = case["op"]
    if op == "plan":
        ctx, new = _plan_lengths(case)
        ps = case["page"]
        pages = sum(-(-(c + n) // ps) - -(-c // ps) for c, n in zip(ctx, new))
        return {"bytes": 16 * len(ctx) + 8 * sum(new) + 8 * pages, "flops": sum(new)}
    d, hq, hkv = case["dim"], case["heads"], case["kv_heads"]
    if op == "shared":
        size, prefix, new, keys = _shared_lengths(case)
        T, pairs, seen, b = sum(new), 0, sum(prefix), 0
        for n, p in zip(size, prefix):
            for i in range(b, b + n):
                pairs += new[i] * (keys[i] - new[i]) + new[i] * (new[i] + 1) // 2
                seen += keys[i] - p
            b += n
        return {"bytes": 4 * seen * hkv * d + T * hq * (4 * d + 4), "flops": 4 * d * hq * pairs}
    T, rows = case["tokens"], hq + hkv
    tables = 4 * T * (case["rotary"] + case["axes"])
    if op == "rope":
        return {"bytes": 4 * T * rows * d + tables, "flops": 8 * T * rows * d}
    if op == "ropegrad":
        return {"bytes": 6 * T * rows * d + tables, "flops": 16 * T * rows * d}
    return {"bytes": 4 * T * (rows + hkv) * d + tables + 4 * T, "flops": 8 * T * rows * d}


# ---- inputs ---------------------------------------------------------------------------------

def _scan(lengths):
    out = [0]
    for n in lengths:
        out.append(out[-1] + n)
    return out


def _ints(x, device="cuda"):
    return torch.tensor(x, dtype=torch.int32, device=device)


def _tables(rows, rot):
    inv = ROTARY_BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    ang = torch.arange(rows, dtype=torch.float64)[:, None] * inv
    return ang.cos().float().cuda(), ang.sin().float().cuda()


def _prepare_plan(case, seed):
    ctx, new = _plan_lengths(case)
    ps = case["page"]
    old = [-(-c // ps) for c in ctx]
    need = sum(-(-(c + n) // ps) for c, n in zip(ctx, new)) - sum(old)
    spare = 7
    num_pages = sum(old) + need + spare
    perm = torch.randperm(num_pages, generator=torch.Generator().manual_seed(seed)).int()
    width = max(1, max(-(-(c + n) // ps) for c, n in zip(ctx, new)))
    table = torch.full((case["batch"], width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(old):
        table[b, :n] = perm[at:at + n]
        at += n
    free = torch.full((num_pages,), -1, dtype=torch.int32)
    free[:need + spare] = perm[at:]
    return {"case": case, "ctx": _ints(ctx), "new": _ints(new), "table": table.cuda(),
            "free": free.cuda(), "count": _ints([need + spare]), "total": sum(new),
            "num_pages": num_pages}


def _prepare_rope(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T, hq, hkv, d, rot = (case[k] for k in ("tokens", "heads", "kv_heads", "dim", "rotary"))

    def rows(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)

    # heads of different sizes, a few large components
    x = torch.randn((T, hq + 2 * hkv, d), generator=gen, device="cuda")
    x *= torch.exp2(torch.randn((hq + 2 * hkv, 1), generator=gen, device="cuda").clamp(-3, 3))
    x[..., 5] *= 20
    x = x.to(torch.bfloat16)
    parts = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    q, k, v = parts if case["packed"] else (t.contiguous() for t in parts)
    s = {"case": case, "q": q, "k": k, "v": v, "qw": None, "kw": None}
    if case["norm"]:
        wtype = torch.float32 if case["w32"] else torch.bfloat16
        s["qw"], s["kw"] = ((1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(wtype)
                            for _ in range(2))
    longest = 4096 if case["axes"] == 1 else 512
    s["cos"], s["sin"] = _tables(longest, rot)
    s["pos"] = torch.randint(0, longest, (case["axes"], T), generator=gen, device="cuda",
                             dtype=torch.int32)
    if case["axes"] == 1:
        s["pos"] = (s["pos"][:, :1] + torch.arange(T, device="cuda", dtype=torch.int32)) % longest
    s["pos"] = s["pos"].contiguous()
    s["sections"] = _sections(case) if case["axes"] > 1 else None
    if case["op"] == "ropegrad":
        s["gq"], s["gk"] = rows(T, hq, d), rows(T, hkv, d)
    if case["op"] == "append":
        ps = case["page"]
        pages = -(-T // ps) + 2
        s["kc"], s["vc"] = rows(pages, ps, hkv, d), rows(pages, ps, hkv, d)
        slots = torch.randperm(pages * ps, generator=gen, device="cuda")[:T].int()
        order = torch.randperm(pages, generator=gen, device="cuda").int()
        if T > 256:  # whole runs of slots, page by page
            t = torch.arange(T, device="cuda", dtype=torch.int32)
            slots = order[(t // ps).long()] * ps + t % ps
        slots[T // 2] = -1  # a padded token
        s["slots"] = slots.int().contiguous()
    return s


def _prepare_shared(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    size, prefix, new, keys = _shared_lengths(case)
    d, hq, hkv, ps = (case[k] for k in ("dim", "heads", "kv_heads", "page"))
    starts = _scan(size)
    batch = starts[-1]
    # pages that a prefix fills belong to the whole group, the page that it ends in is copied
    own_pages = []
    for g, p in enumerate(prefix):
        for b in range(starts[g], starts[g + 1]):
            own_pages.append(-(-keys[b] // ps) - p // ps)
    num_pages = sum(p // ps for p in prefix) + sum(own_pages) + 1
    perm = torch.randperm(num_pages, generator=torch.Generator().manual_seed(seed)).int()
    table = torch.full((batch, max(1, max(-(-n // ps) for n in keys))), -1, dtype=torch.int32)
    at = 0
    for g, p in enumerate(prefix):
        whole = perm[at:at + p // ps]
        at += p // ps
        for b in range(starts[g], starts[g + 1]):
            table[b, :p // ps] = whole
            table[b, p // ps:p // ps + own_pages[b]] = perm[at:at + own_pages[b]]
            at += own_pages[b]
    s = {"case": case, "size": size, "prefix": prefix, "new": new, "keys": keys, "starts": starts,
         "table": table.cuda(), "seqlens": _ints(keys), "group_starts": _ints(starts),
         "prefix_lens": _ints(prefix), "scale": d ** -0.5, "max_q": max(new)}
    s["cu"] = None if case["new_lo"] == case["new_hi"] == 1 else _ints(_scan(new))
    for name in ("kc", "vc"):
        s[name] = torch.empty((num_pages, ps, hkv, d), dtype=torch.bfloat16, device="cuda")
        step = max(1, (1 << 26) // (ps * hkv * d))
        for i in range(0, num_pages, step):
            x = torch.randn((min(step, num_pages - i), ps, hkv, d), generator=gen, device="cuda")
            s[name][i:i + step] = x.to(torch.bfloat16)
    for g, p in enumerate(prefix):  # the copies of the page that the prefix ends in
        if p % ps:
            j = table[starts[g]:starts[g + 1], p // ps].long().cuda()
            for name in ("kc", "vc"):
                s[name][j, :p % ps] = s[name][j[0], :p % ps]
    s["q"] = (1.5 * torch.randn((sum(new), hq, d), generator=gen, device="cuda")).to(torch.bfloat16)
    return s


def prepare(case, seed):
    if case["op"] == "plan":
        return _prepare_plan(case, seed)
    return _prepare_shared(case, seed) if case["op"] == "shared" else _prepare_rope(case, seed)


# ---- the plain form ---------------------------------------------------------------------------

def _plain_plan(s):
    ps = s["case"]["page"]
    ctx, new = s["ctx"].long(), s["new"].long()
    cu = torch.cat((ctx.new_zeros(1), new.cumsum(0)))
    old = (ctx + ps - 1) // ps
    need = (ctx + new + ps - 1) // ps - old
    first = need.cumsum(0) - need
    t = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    pos = ctx[b] + t - cu[b]
    taken = s["count"].long() - 1 - (first[:, None] + torch.arange(s["table"].shape[1], device="cuda")
                                     - old[:, None])
    j = torch.arange(s["table"].shape[1], device="cuda")
    fresh = (j >= old[:, None]) & (j < (old + need)[:, None])
    table = torch.where(fresh, s["free"][taken.clamp(0, s["free"].shape[0] - 1)], s["table"])
    s["table"].copy_(table)
    slots = table[b, pos // ps].long() * ps + pos % ps
    return {"table": s["table"], "cu": cu.int(), "after": (ctx + new).int(), "positions": pos.int(),
            "slots": slots.int(), "left": s["count"] - need.sum().int()}


def _plain_angles(s):
    """cos and sin of every token's planes [T, 1, rotary / 2]."""
    axis = torch.tensor(_plane_axis(s["case"]), device="cuda")
    plane = torch.arange(axis.shape[0], device="cuda")
    row = s["pos"].long()[axis].t()
    return s["cos"][row, plane][:, None], s["sin"][row, plane][:, None]


def _split(x, rot, interleaved):
    half = rot // 2
    if interleaved:
        return x[..., 0:rot:2], x[..., 1:rot:2]
    return x[..., :half], x[..., half:rot]


def _join(a, b, rest, interleaved):
    turned = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((turned, rest), -1)


def _plain_rows(s, x, w, cos, sin):
    c = s["case"]
    x = x.float()
    if w is not None:
        x = x * ((x * x).mean(-1, keepdim=True) + EPS) ** -0.5 * w.float()
    a, b = _split(x, c["rotary"], c["interleaved"])
    return _join(a * cos - b * sin, a * sin + b * cos, x[..., c["rotary"]:],
                 c["interleaved"]).to(torch.bfloat16)


def _plain_rows_grad(s, g, x, w, cos, sin):
    c = s["case"]
    g, x = g.float(), x.float()
    a, b = _split(g, c["rotary"], c["interleaved"])
    g = _join(a * cos + b * sin, b * cos - a * sin, g[..., c["rotary"]:], c["interleaved"])
    if w is None:
        return g.to(torch.bfloat16), None
    r = ((x * x).mean(-1, keepdim=True) + EPS) ** -0.5
    n = x * r
    dw = (n * g).sum((0, 1))
    g = g * w.float()
    return (r * (g - n * (n * g).mean(-1, keepdim=True))).to(torch.bfloat16), dw


def _plain_rope(s):
    cos, sin = _plain_angles(s)
    if s["case"]["op"] == "ropegrad":
        dq, dqw = _plain_rows_grad(s, s["gq"], s["q"], s["qw"], cos, sin)
        dk, dkw = _plain_rows_grad(s, s["gk"], s["k"], s["kw"], cos, sin)
        return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}
    q, k = _plain_rows(s, s["q"], s["qw"], cos, sin), _plain_rows(s, s["k"], s["kw"], cos, sin)
    if s["case"]["op"] == "rope":
        return {"q": q, "k": k}
    at = torch.nonzero(s["slots"] >= 0)[:, 0]
    slot = s["slots"][at].long()
    s["kc"].flatten(0, 1)[slot] = k[at]
    s["vc"].flatten(0, 1)[slot] = s["v"][at]
    return {"q": q, "k_cache": s["kc"], "v_cache": s["vc"]}


def _gather(s, cache, rows, lo, hi):
    """fp32 keys [rows, hi - lo, Hkv, d] at positions lo .. hi - 1 through the table."""
    ps = s["case"]["page"]
    j = torch.arange(lo, hi, device="cuda")
    return cache[s["table"][rows][:, j // ps].clamp(min=0).long(), j % ps].float()


def _plain_part(q, k, v, seen):
    """Maximum, sum and weighted values of q [B, Hkv, R, d] over keys [B, L, Hkv, d]."""
    x = q @ k.permute(0, 2, 3, 1)
    if seen is not None:
        x.masked_fill_(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    v = torch.where((torch.ones_like(x[:, :1, :1]) if seen is None else seen.any(2, keepdim=True).float())
                    .permute(0, 3, 1, 2) > 0, v, 0.0)
    return m, x.sum(-1, keepdim=True), x @ v.permute(0, 2, 1, 3)


def _plain_shared(s):
    c = s["case"]
    d, hq, hkv = c["dim"], c["heads"], c["kv_heads"]
    cu = _scan(s["new"])
    out, lse = [], []
    for g, p in enumerate(s["prefix"]):
        b0, b1 = s["starts"][g], s["starts"][g + 1]
        n, longest, widest = b1 - b0, max(s["keys"][b0:b1]), max(s["new"][b0:b1])
        rows = torch.arange(b0, b1, device="cuda")
        new = _ints(s["new"][b0:b1])[:, None]
        i = torch.arange(widest, device="cuda")
        real = i < new
        at = (_ints(cu[b0:b1])[:, None] + i).clamp(max=cu[-1] - 1)
        q = s["q"][at.long()].float() * s["scale"]  # [n, widest, Hq, d]
        q = q.view(n, widest, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d)
        first = rows[:1]
        k, v = _gather(s, s["kc"], first, 0, p), _gather(s, s["vc"], first, 0, p)
        m, l, o = _plain_part(q.transpose(0, 1).reshape(1, hkv, -1, d), k, v, None)
        m, l, o = (x.view(hkv, n, -1, x.shape[-1]).transpose(0, 1) for x in (m, l, o))
        if longest > p:
            k, v = _gather(s, s["kc"], rows, p, longest), _gather(s, s["vc"], rows, p, longest)
            keys = s["seqlens"][b0:b1, None]
            last = keys - new + i  # the position of each query
            seen = torch.arange(p, longest, device="cuda") <= torch.where(real, last, -1)[..., None]
            seen = seen.repeat(1, hq // hkv, 1)[:, None]
            m2, l2, o2 = _plain_part(q, k, v, seen)
            top = torch.maximum(m, m2)
            w, w2 = (m - top).exp(), (m2 - top).exp()
            m, l, o = top, l * w + l2 * w2, o * w + o2 * w2
        o = (o / l).view(n, hkv, hq // hkv, widest, d).permute(0, 3, 1, 2, 4)
        ls = (m + l.log()).view(n, hkv, hq // hkv, widest).permute(0, 3, 1, 2)
        out.append(o.reshape(n, widest, hq, d)[real].to(torch.bfloat16))
        lse.append(ls.reshape(n, widest, hq)[real])
    lse = torch.cat(lse)
    return {"out": torch.cat(out), "lse": lse if s["cu"] is None else lse.t().contiguous()}


def _plain(s):
    op = s["case"]["op"]
    return _plain_plan(s) if op == "plan" else _plain_shared(s) if op == "shared" else _plain_rope(s)


# ---- the framework's calls ---------------------------------------------------------------------

def _own(s):
    from exact_attention_70_gb300 import binding
    c = s["case"]
    if c["op"] == "plan":
        cu, after, positions, slots, left = binding.attn_kvcache_plan(
            s["ctx"], s["new"], s["table"], s["free"], s["count"], c["page"], s["num_pages"],
            s["total"])
        return {"table": s["table"], "cu": cu, "after": after, "positions": positions,
                "slots": slots, "left": left}
    if c["op"] == "shared":
        out, lse = binding.attn_decode_kvcache_shared(
            s["q"], s["kc"], s["vc"], s["seqlens"], s["table"], s["group_starts"],
            s["prefix_lens"], s["cu"], s["max_q"], s["scale"])
        return {"out": out, "lse": lse}
    how = dict(q_weight=s["qw"], k_weight=s["kw"], eps=EPS, rotary_cos=s["cos"],
               rotary_sin=s["sin"], positions=s["pos"], rotary_interleaved=c["interleaved"],
               sections=s["sections"], sections_interleaved=c["mixed"])
    if c["op"] == "rope":
        q, k = binding.attn_qk_norm_rope(s["q"], s["k"], **how)
        return {"q": q, "k": k}
    if c["op"] == "ropegrad":
        dq, dk, dqw, dkw = binding.attn_qk_norm_rope_bwd(s["gq"], s["gk"], s["q"], s["k"], **how)
        return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}
    q = binding.attn_kvcache_append_norm_rope(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["slots"],
                                              **how)
    return {"q": q, "k_cache": s["kc"], "v_cache": s["vc"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---- the definition in 64 bits -------------------------------------------------------------------

def _exact_plan(s):
    """Token by token on the host."""
    ps = s["case"]["page"]
    table, free = s["table"].tolist(), s["free"].tolist()
    left = s["count"].item()
    cu, after, positions, slots = [0], [], [], []
    for b, (c, n) in enumerate(zip(s["ctx"].tolist(), s["new"].tolist())):
        for p in range(c, c + n):
            if p % ps == 0:
                left -= 1
                table[b][p // ps] = free[left]
            positions.append(p)
            slots.append(table[b][p // ps] * ps + p % ps)
        cu.append(cu[-1] + n)
        after.append(c + n)
    return {"table": _ints(table), "cu": _ints(cu), "after": _ints(after),
            "positions": _ints(positions), "slots": _ints(slots), "left": _ints([left])}


def _exact_rope(s):
    c = s["case"]
    half, d = c["rotary"] // 2, c["dim"]
    sections = _sections(c)
    # plane by plane: its axis, its two components, its turn as a complex number per token
    lead = []
    left = list(sections)
    for i in range(half):
        if c["axes"] == 1:
            lead.append(0)
        elif c["mixed"]:
            a = i % c["axes"]
            lead.append(a if a and left[a] > 0 else 0)
            left[lead[-1]] -= 1
        else:
            a = 0
            while i >= sum(sections[:a + 1]):
                a += 1
            lead.append(a)
    ia = [2 * i if c["interleaved"] else i for i in range(half)]
    ib = [2 * i + 1 if c["interleaved"] else i + half for i in range(half)]
    row = torch.stack([s["pos"][a].long() for a in lead], 1)
    cols = torch.arange(half, device="cuda")
    turn = torch.complex(s["cos"].double()[row, cols], s["sin"].double()[row, cols])[:, None]

    def rotated(x, w):
        x = x.clone()
        z = torch.complex(x[..., ia], x[..., ib]) * w
        x[..., ia], x[..., ib] = z.real, z.imag
        return x

    def normed(x, w):
        return x if w is None else x / torch.sqrt(x.square().sum(-1, keepdim=True) / d + EPS) * w

    def weight(w):
        return None if w is None else w.double()

    if c["op"] == "ropegrad":
        got = {}
        for name, x, g, w in (("q", s["q"], s["gq"], s["qw"]), ("k", s["k"], s["gk"], s["kw"])):
            back = rotated(g.double(), turn.conj())
            x, w = x.double(), weight(w)
            if w is None:
                got["d" + name], got["d%s_weight" % name] = back, None
                continue
            norm = torch.sqrt(x.square().sum(-1, keepdim=True) / d + EPS)
            got["d%s_weight" % name] = torch.einsum("thd,thd->d", back, x / norm)
            inner = (back * w * x).sum(-1, keepdim=True)
            got["d" + name] = back * w / norm - x * inner / (d * norm ** 3)
        return got
    q = rotated(normed(s["q"].double(), weight(s["qw"])), turn)
    k = rotated(normed(s["k"].double(), weight(s["kw"])), turn)
    if c["op"] == "rope":
        return {"q": q, "k": k}
    kc, vc = s["kc"].double(), s["vc"].double()
    slots = s["slots"].long()
    at = torch.arange(slots.shape[0], device="cuda")[slots >= 0]
    ps = c["page"]
    kc[slots[at] // ps, slots[at] % ps] = k[at]
    vc[slots[at] // ps, slots[at] % ps] = s["v"][at].double()
    return {"q": q, "k_cache": kc, "v_cache": vc}


def _exact_shared(s):
    """Sequence by sequence, each over all its keys through its own row of the table."""
    c = s["case"]
    d, hq, hkv, ps = c["dim"], c["heads"], c["kv_heads"], c["page"]
    g, t = hq // hkv, 0
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    for b, (n, L) in enumerate(zip(s["new"], s["keys"])):
        if n == 0:
            continue
        p = torch.arange(L, device="cuda")
        page = s["table"][b].long()[p // ps]
        seen = p <= torch.arange(L - n, L, device="cuda")[:, None]
        for h in range(hkv):
            k, v = s["kc"][page, p % ps, h].double(), s["vc"][page, p % ps, h].double()
            q = s["q"][t:t + n, h * g:(h + 1) * g].double() * s["scale"]
            x = torch.einsum("tgd,kd->tgk", q, k).masked_fill(~seen[:, None], -math.inf)
            e = torch.logsumexp(x, -1)
            out[t:t + n, h * g:(h + 1) * g] = torch.einsum("tgk,kd->tgd", (x - e[..., None]).exp(), v)
            lse[t:t + n, h * g:(h + 1) * g] = e
        t += n
    return {"out": out, "lse": lse if s["cu"] is None else lse.t().contiguous()}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    return _exact_plan(s) if op == "plan" else _exact_shared(s) if op == "shared" else _exact_rope(s)
