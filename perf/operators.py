"""The operators of the 8-bit paged KV cache as a user calls them, and their plain form.

The cache: k_cache, v_cache uint8 e4m3 codes [num_pages, page_size, Hkv, d]; k_scale, v_scale uint8
[num_pages, Hkv, page_size], byte b standing for 2^(b - 127), one per (token, kv head).  A row x is
stored with e = the smallest integer >= -126 with max|x| <= 448 2^e, b = e + 127 and the codes
e4m3(x 2^-e) (nearest, ties to even).

  append  new keys (rotated) and values written into the cache
  decode  one query token per sequence over the cache
  read    the cache back as packed bf16 keys and values
  chunk   append, then attention of the chunk's query tokens over cache and chunk
"""
import math
import random

import torch

own = False

SCALE_BIAS = 127
ROTARY_BASE = 10000.0


# ---- cases ---------------------------------------------------------------------------------
# q: new tokens per sequence (lo, hi), ctx: tokens already in the cache (lo, hi); a sequence's
# lengths come from the case alone ("lens"), the values and the order of the pages from the seed.

def _case(name, op, batch, q, ctx, heads, kv_heads, dim, page, rotary=0, interleaved=False,
          window=-1, lens=1):
    return {"name": name, "op": op, "batch": batch, "q_lo": q[0], "q_hi": q[1],
            "ctx_lo": ctx[0], "ctx_hi": ctx[1], "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "page": page, "rotary": rotary, "interleaved": interleaved, "window": window,
            "lens": lens}


def listed():
    return [
        # the cache write of one generation step of 64 sequences: latency
        _case("append-step", "append", 64, (1, 1), (64, 512), 32, 8, 128, 256, rotary=128, lens=11),
        # a few ragged prompts, small heads, part of the head rotated in interleaved planes
        _case("append-ragged", "append", 11, (1, 700), (0, 900), 6, 3, 64, 16, rotary=32,
              interleaved=True, lens=12),
        # the cache write of a chunked-prefill step: 8 sequences of 2048 new tokens
        _case("append-prompt", "append", 8, (2048, 2048), (2048, 16384), 32, 8, 128, 256,
              rotary=128, lens=13),
        # one short conversation: the smallest decode, latency
        _case("decode-one", "decode", 1, (1, 1), (700, 701), 8, 2, 64, 64, lens=14),
        # many short sequences (empty ones among them), 7 query heads a kv head, small pages
        _case("decode-ragged", "decode", 37, (1, 1), (0, 3000), 14, 2, 128, 16, lens=15),
        # two long documents: few rows, a long axis to split
        _case("decode-long", "decode", 2, (1, 1), (100001, 131071), 32, 8, 128, 256, lens=16),
        # a full serving batch of 1K to 32K tokens each
        _case("decode-batch", "decode", 64, (1, 1), (1024, 32768), 32, 8, 128, 256, lens=17),
        # a small cache handed on (a few short sequences)
        _case("read-short", "read", 3, (1, 1), (1, 600), 4, 2, 64, 32, lens=18),
        # prefixes of a serving batch read back for a step on bf16 keys and values
        _case("read-long", "read", 8, (1, 1), (8192, 32768), 32, 8, 128, 256, lens=19),
        # checking 4 drafted tokens of each of 16 sequences
        _case("chunk-verify", "chunk", 16, (4, 4), (1024, 8192), 32, 8, 128, 64, rotary=128,
              lens=20),
        # a mixed step with a sliding window: one token to some hundred, d = 64
        _case("chunk-window", "chunk", 5, (1, 600), (0, 5000), 16, 4, 64, 128, rotary=32,
              interleaved=True, window=1024, lens=21),
        # a chunked-prefill step over long prefixes
        _case("chunk-prefill", "chunk", 8, (2048, 2048), (2048, 16384), 32, 8, 128, 256,
              rotary=128, lens=22),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "read", "chunk"])
    dim = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128, 256])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8])
    rotary = rng.choice([0, 16, dim // 2, dim]) if op in ("append", "chunk") else 0
    c = _case("", op, 1, (1, 1), (0, 1), heads, kv_heads, dim, page, rotary=rotary,
              interleaved=rng.random() < 0.5, lens=rng.randrange(1 << 30))
    del c["name"]
    if op == "append":
        total = _log_int(rng, 1, 16000)
        c["batch"] = min(total, _log_int(rng, 1, 128))
        c["q_hi"] = max(1, total // c["batch"])
        c["q_lo"] = rng.randint(0, c["q_hi"])
        c["ctx_hi"] = _log_int(rng, 1, 12000) if c["batch"] <= 16 else _log_int(rng, 1, 1000)
    elif op in ("decode", "read"):
        total = _log_int(rng, 32, 1000000 if op == "decode" else 160000)
        c["batch"] = min(total, _log_int(rng, 1, 128))
        c["ctx_hi"] = min(131071, max(1, total // c["batch"]))
        c["ctx_lo"] = rng.randint(0, c["ctx_hi"])
    else:
        c["batch"] = _log_int(rng, 1, 16)
        c["q_hi"] = _log_int(rng, 1, 4000 // c["batch"])
        c["q_lo"] = rng.randint(1, c["q_hi"])
        c["ctx_hi"] = _log_int(rng, 1, 16000)
        c["window"] = rng.choice([-1, -1, rng.randint(1, 4096)])
    return c


def _lengths(case):
    r = random.Random(case["lens"])
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]
    new = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["batch"])]
    return [max(1, ctx[0])] + ctx[1:], [max(1, new[0])] + new[1:]


def _pairs(ctx, new, window):
    """Visible (query, key) pairs: query i sits at key position ctx + i, sees `window` before it."""
    total = 0
    for c, n in zip(ctx, new):
        if window < 0:
            total += n * c + n * (n + 1) // 2
        else:
            total += sum(min(c + i + 1, window + 1) for i in range(n))
    return total


def work(case):
    ctx, new = _lengths(case)
    d, hq, hkv, rot = case["dim"], case["heads"], case["kv_heads"], case["rotary"]
    T = sum(new)
    write = T * hkv * 2 * (2 * d + d + 1) + T * rot * 4 + 4 * T  # bf16 in, codes and scales out, tables
    rotate = 3 * T * hkv * rot
    if case["op"] == "append":
        return {"bytes": write, "flops": rotate + 2 * T * hkv * d}
    if case["op"] == "decode":
        return {"bytes": sum(ctx) * hkv * 2 * (d + 1) + case["batch"] * hq * (4 * d + 4),
                "flops": 4 * d * hq * sum(ctx)}
    if case["op"] == "read":
        return {"bytes": sum(ctx) * hkv * 2 * (d + 1 + 2 * d), "flops": 2 * sum(ctx) * hkv * d}
    # a windowed row does not need the prefix before its window
    w = case["window"]
    seen = sum(c if w < 0 else min(c, w) for c, n in zip(ctx, new) if n)
    return {"bytes": write + seen * hkv * 2 * (d + 1) + T * hq * (4 * d + 4),
            "flops": rotate + 3 * T * hq * rot + 4 * d * hq * _pairs(ctx, new, w)}


# ---- inputs ---------------------------------------------------------------------------------

def _cu(lengths, device):
    out = [0]
    for n in lengths:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device=device)


def _filled(shape, gen, device):
    """Codes and scale bytes of N(0, 1) rows, their size varying from row to row."""
    P, ps, H, d = shape
    codes = torch.empty(shape, dtype=torch.uint8, device=device)
    scale = torch.empty((P, H, ps), dtype=torch.uint8, device=device)
    step = max(1, (1 << 26) // (ps * H * d))
    for a in range(0, P, step):
        n = min(step, P - a)
        x = torch.randn((n, ps, H, d), generator=gen, device=device)
        x *= torch.exp2(0.5 * torch.randn((n, ps, H, 1), generator=gen, device=device).clamp(-2, 2))
        m, e = torch.frexp(x.abs().amax(-1))
        e = e - 9 + (m > 0.875).to(e.dtype)
        codes[a:a + n] = (x * torch.exp2(-e.float())[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scale[a:a + n] = (e + SCALE_BIAS).to(torch.uint8).transpose(1, 2)
    return codes, scale


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    ctx, new = _lengths(case)
    d, hq, hkv, ps = case["dim"], case["heads"], case["kv_heads"], case["page"]
    op = case["op"]
    lens = [c + n for c, n in zip(ctx, new)] if op in ("append", "chunk") else ctx
    pages = [(n + ps - 1) // ps for n in lens]
    num_pages = max(1, sum(pages)) + 1
    perm = torch.randperm(num_pages, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((case["batch"], max(1, max(pages))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
        at += n

    def rows(*shape):
        return torch.randn(shape, generator=gen, device=dev).to(torch.bfloat16)

    s = {"case": case, "ctx": ctx, "new": new, "table": table.to(dev),
         "seqlens": torch.tensor(ctx, dtype=torch.int32, device=dev),
         "longest": max([1] + lens), "scale": d ** -0.5}
    s["kc"], s["ks"] = _filled((num_pages, ps, hkv, d), gen, dev)
    s["vc"], s["vs"] = _filled((num_pages, ps, hkv, d), gen, dev)
    T = sum(new)
    if op in ("append", "chunk"):
        s["cu"] = _cu(new, dev)
        s["k"], s["v"] = rows(T, hkv, d), rows(T, hkv, d)
        s["max_q"], s["total_k"] = max(new), sum(lens)
        s["cos"] = s["sin"] = None
        if case["rotary"]:
            rot = case["rotary"]
            inv = ROTARY_BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
            ang = torch.arange(s["longest"], dtype=torch.float64)[:, None] * inv
            s["cos"], s["sin"] = ang.cos().float().to(dev), ang.sin().float().to(dev)
    if op == "chunk":
        s["q"] = rows(T, hq, d)
    if op == "decode":
        s["q"] = rows(case["batch"], hq, d)
    if op == "read":
        s["cu"], s["total_k"] = _cu(ctx, dev), sum(ctx)
    return s


# ---- the plain form ---------------------------------------------------------------------------

def _rotated(x, pos, cos, sin, interleaved):
    """x [T, H, d] in its own precision, rows at positions pos."""
    if cos is None:
        return x
    half = cos.shape[1]
    c, s = cos[pos].to(x.dtype)[:, None], sin[pos].to(x.dtype)[:, None]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack((a * c - b * s, a * s + b * c), -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat((a * c - b * s, a * s + b * c), -1)
    return torch.cat((turned, x[..., 2 * half:]), -1)


def _pow2(e):
    """2^e in fp64, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _scale_of(byte):
    """2^(b - 127) in fp32, from its bits (b from 1 on)."""
    return (byte.int() << 23).view(torch.float32)


def _quantised(x):
    """Codes and scale bytes of fp64 rows."""
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m == 0, -126, (e - 9 + (m > 0.875).to(e.dtype)).clamp(min=-126))
    y = x * _pow2(-e)[..., None]
    step = torch.frexp(y)[1].clamp(min=-5) - 4  # 3 bits behind the leading one, down to 2^-9
    code = torch.round(y * _pow2(-step)) * _pow2(step)
    return code.float().to(torch.float8_e4m3fn).view(torch.uint8), (e + SCALE_BIAS).to(torch.uint8)


def _plain_append(s):
    c = s["case"]
    t = torch.arange(s["k"].shape[0], device="cuda")
    b = torch.searchsorted(s["cu"], t, right=True, out_int32=False) - 1
    pos = s["seqlens"][b].long() + t - s["cu"][b]
    page, slot = s["table"][b, pos // c["page"]].long(), pos % c["page"]
    k = _rotated(s["k"].double(), pos, s["cos"], s["sin"], c["interleaved"])
    kq, ks = _quantised(k)
    vq, vs = _quantised(s["v"].double())
    s["kc"][page, slot], s["vc"][page, slot] = kq, vq
    s["ks"][page, :, slot], s["vs"][page, :, slot] = ks, vs
    return pos


def _cached(s, codes, scale, lens):
    """fp32 rows [batch, longest, Hkv, d], zero behind each sequence."""
    ps = s["case"]["page"]
    j = torch.arange(s["longest"], device="cuda")
    page = s["table"][:, j // ps].clamp(min=0).long()
    slot = (j % ps).expand_as(page)
    x = codes[page, slot].view(torch.float8_e4m3fn).float()
    x *= _scale_of(scale[page, :, slot])[..., None]
    return torch.where((j < lens[:, None])[..., None, None], x, 0.0)


def _plain_attention(q, k, v, first, lens, scale, window):
    """q [batch, Lq, Hq, d] at key positions first + i; k, v [batch, Lk, Hkv, d]; fp32."""
    B, Lq, Hq, d = q.shape
    Hkv = k.shape[2]
    qg = q.view(B, Lq, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, d)
    p = (qg * scale) @ k.permute(0, 2, 3, 1)
    j = torch.arange(k.shape[1], device="cuda")
    at = first[:, None, None] + torch.arange(Lq, device="cuda")[:, None]
    seen = (j <= at) & (j < lens[:, None, None])
    if window >= 0:
        seen &= j >= at - window
    p = p.view(B, Hkv, Hq // Hkv, Lq, -1)
    p.masked_fill_(~seen[:, None, None], -math.inf)
    m = p.amax(-1, keepdim=True)
    p.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    l = p.sum(-1, keepdim=True)
    o = p.view(B, Hkv, -1, k.shape[1]) @ v.permute(0, 2, 1, 3)
    o = o.view(B, Hkv, Hq // Hkv, Lq, d) / torch.where(l == 0, 1.0, l)
    lse = (m + l.log())[..., 0]
    return o.permute(0, 3, 1, 2, 4).reshape(B, Lq, Hq, d), lse.permute(0, 3, 1, 2).reshape(B, Lq, Hq)


def _plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "append":
        _plain_append(s)
        return _cache(s)
    if op == "decode":
        lens = s["seqlens"]
        k, v = _cached(s, s["kc"], s["ks"], lens), _cached(s, s["vc"], s["vs"], lens)
        o, lse = _plain_attention(s["q"].float()[:, None], k, v, lens - 1, lens, s["scale"], -1)
        return {"out": o[:, 0].to(torch.bfloat16), "lse": lse[:, 0]}
    if op == "read":
        t = torch.arange(s["total_k"], device="cuda")
        b = torch.searchsorted(s["cu"], t, right=True) - 1
        j = t - s["cu"][b]
        page, slot = s["table"][b, j // c["page"]].long(), j % c["page"]
        k, v = ((x[page, slot].view(torch.float8_e4m3fn).float()
                 * _scale_of(e[page, :, slot])[..., None]).to(torch.bfloat16)
                for x, e in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
        return {"k": k, "v": v}
    pos = _plain_append(s)
    new = s["cu"][1:] - s["cu"][:-1]
    lens = s["seqlens"] + new
    k, v = _cached(s, s["kc"], s["ks"], lens), _cached(s, s["vc"], s["vs"], lens)
    q = _rotated(s["q"].float(), pos, s["cos"], s["sin"], c["interleaved"])
    i = torch.arange(s["max_q"], device="cuda")
    row = (s["cu"][:-1, None] + i).clamp(max=q.shape[0] - 1)
    o, lse = _plain_attention(q[row], k, v, s["seqlens"], lens, s["scale"], c["window"])
    real = i < new[:, None]
    return {"out": o[real].to(torch.bfloat16), "lse": lse[real].t().contiguous(), **_cache(s)}


def _cache(s):
    """The updated cache: codes as the values they stand for, scale bytes as they are."""
    f8 = torch.float8_e4m3fn
    return {"k_cache": s["kc"].view(f8), "v_cache": s["vc"].view(f8), "k_scale": s["ks"],
            "v_scale": s["vs"]}


# ---- the framework's calls ---------------------------------------------------------------------

def _own(s):
    from exact_attention_70_gb300 import binding
    c, op = s["case"], s["case"]["op"]
    cache = (s["kc"], s["vc"], s["ks"], s["vs"])
    if op == "append":
        binding.attn_kvcache_append_fp8(s["k"], s["v"], *cache, s["seqlens"], s["table"], s["cu"],
                                        s["cos"], s["sin"], c["interleaved"])
        return _cache(s)
    if op == "decode":
        out, lse = binding.attn_decode_kvcache_fp8(s["q"], *cache, s["seqlens"], s["table"],
                                                   s["scale"])
        return {"out": out, "lse": lse}
    if op == "read":
        k, v = binding.attn_kvcache_read_fp8(*cache, s["table"], s["cu"], s["total_k"])
        return {"k": k, "v": v}
    out, lse = binding.attn_fwd_kvcache_fp8(
        s["q"], s["k"], s["v"], *cache, s["seqlens"], s["table"], s["cu"], s["max_q"],
        s["total_k"], s["scale"], True, c["window"], -1, s["cos"], s["sin"], c["interleaved"])
    return {"out": out, "lse": lse, **_cache(s)}


def run(state):
    return _own(state) if own else _plain(state)


# ---- the definition in 64 bits -------------------------------------------------------------------

def _grid():
    """The non-negative e4m3 values by code."""
    return torch.tensor([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10)
                         for c in range(127)], dtype=torch.float64, device="cuda")


def _powers():
    """2^(b - 127) by scale byte."""
    return torch.tensor([2.0 ** (b - SCALE_BIAS) for b in range(256)], dtype=torch.float64,
                        device="cuda")


def _exact_row(x, grid):
    """Nearest grid values (ties to the even code) and exponents of rows x [..., d]."""
    top = x.abs().amax(-1)
    e = torch.full(top.shape, -126.0, dtype=torch.float64, device=x.device)
    for k in range(40, -127, -1):  # the smallest exponent that holds the row
        e = torch.where(top <= 448.0 * 2.0 ** k, float(k), e)
    y = (x / _powers()[(e + SCALE_BIAS).long()][..., None]).abs()
    hi = torch.searchsorted(grid, y.contiguous()).clamp(1, 126)
    up, down = grid[hi] - y, y - grid[hi - 1]
    pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)
    return torch.where(x < 0, -grid[pick], grid[pick]), e


def exact(case, seed):
    if 4 * case["dim"] * case["heads"] * _pairs(*_lengths(case), case["window"]) > 8e12:
        return None
    s = prepare(case, seed)
    op, ps, d = case["op"], case["page"], case["dim"]
    hq, hkv = case["heads"], case["kv_heads"]
    grid = _grid()
    value = torch.cat((grid, grid[:1], -grid, grid[:1]))
    powers = _powers()
    kc, vc = value[s["kc"].long()], value[s["vc"].long()]
    ke, ve = s["ks"].double() - SCALE_BIAS, s["vs"].double() - SCALE_BIAS
    half = case["rotary"] // 2

    def turn(x, p):  # x [n, H, d] at positions p, plane by plane as complex numbers
        if not half:
            return x
        w = torch.complex(s["cos"][p].double(), s["sin"][p].double())[:, None]
        x = x.clone()
        a, b = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if case["interleaved"]
                else (slice(0, half), slice(half, 2 * half)))
        z = torch.complex(x[..., a], x[..., b]) * w
        x[..., a], x[..., b] = z.real, z.imag
        return x

    outs, lses, ks, vs = [], [], [], []
    t0 = 0
    for b in range(case["batch"]):
        table = s["table"][b].long()
        L, n = s["ctx"][b], s["new"][b] if op in ("append", "chunk") else 0
        if n:
            p = torch.arange(L, L + n, device="cuda")
            page, slot = table[p // ps], p % ps
            for x, c, e in ((turn(s["k"][t0:t0 + n].double(), p), kc, ke),
                            (s["v"][t0:t0 + n].double(), vc, ve)):
                c[page, slot], e[page, :, slot] = _exact_row(x, grid)
            L += n
        if op != "append":
            p = torch.arange(L, device="cuda")
            page, slot = table[p // ps], p % ps
            k = kc[page, slot] * powers[(ke[page, :, slot] + SCALE_BIAS).long()][..., None]
            v = vc[page, slot] * powers[(ve[page, :, slot] + SCALE_BIAS).long()][..., None]
            if op == "read":
                ks.append(k)
                vs.append(v)
            else:
                if op == "decode":
                    q, i = s["q"][b:b + 1].double(), p.new_full((1,), L - 1)
                else:
                    i = torch.arange(L - n, L, device="cuda")
                    q = turn(s["q"][t0:t0 + n].double(), i)
                seen = p <= i[:, None]
                if case["window"] >= 0:
                    seen &= p >= i[:, None] - case["window"]
                for h in range(hkv):
                    g = hq // hkv
                    S = torch.einsum("tgd,kd->tgk", q[:, h * g:(h + 1) * g], k[:, h]) * s["scale"]
                    S = S.masked_fill(~seen[:, None], -math.inf)
                    lse = torch.logsumexp(S, -1) if L else S.new_full(S.shape[:2], -math.inf)
                    w = torch.exp(S - torch.where(lse == -math.inf, 0.0, lse)[..., None])
                    outs.append((t0, h, torch.einsum("tgk,kd->tgd", w, v[:, h])))
                    lses.append((t0, h, lse))
        t0 += n if op != "decode" else 1
    if op == "read":
        return {"k": torch.cat(ks), "v": torch.cat(vs)}
    got = {}
    if op != "append":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
        g = hq // hkv
        for (t, h, o), (_, _, l) in zip(outs, lses):
            out[t:t + o.shape[0], h * g:(h + 1) * g] = o
            lse[t:t + o.shape[0], h * g:(h + 1) * g] = l
        got = {"out": out, "lse": lse if op == "decode" else lse.t().contiguous()}
    if op != "decode":
        got |= {"k_cache": kc, "v_cache": vc, "k_scale": (ke + SCALE_BIAS).to(torch.uint8),
                "v_scale": (ve + SCALE_BIAS).to(torch.uint8)}
    return got
