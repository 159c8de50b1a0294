"""The calls of a step around paged attention (page plan, norm with rotation, decode behind shared
prefixes) restated in 64 bits, on the CPU, with the error bounds that the kernels' roundings allow.

A rounding to bf16 is off by at most 2^-8 of the value (half a step), or by half of the smallest
subnormal, 2^-134."""
import math
from dataclasses import dataclass

import torch

BF16 = 2.0 ** -8
TINY = 2.0 ** -133


# ---- page plan -------------------------------------------------------------------------------

def plan(cache_seqlens, new_lens, table, free, count, page_size, total):
    """Lists (table, cu, after, positions, slots, left), token by token."""
    table = [list(r) for r in table]
    left, cu, positions, slots = count, [0], [], []
    for b, (c, n) in enumerate(zip(cache_seqlens, new_lens)):
        for p in range(c, c + n):
            if p % page_size == 0:
                left -= 1
                table[b][p // page_size] = free[left]
            positions.append(p)
            slots.append(table[b][p // page_size] * page_size + p % page_size)
        cu.append(cu[-1] + n)
    pad = total - cu[-1]
    return (table, cu, [c + n for c, n in zip(cache_seqlens, new_lens)], positions + [0] * pad,
            slots + [-1] * pad, left)


# ---- norm and rotation -------------------------------------------------------------------------

def plane_axes(half, axes, sections, mixed):
    """The axis of each of `half` planes."""
    if axes == 1:
        return [0] * half
    if not mixed:
        return [a for a in range(axes) for _ in range(sections[a])]
    left, out = list(sections), []
    for i in range(half):
        a = i % axes if left[i % axes] > 0 else 0
        left[a] -= 1
        out.append(a)
    return out


@dataclass
class Turn:
    """The rotation of T tokens: cos and sin [T, 1, half], planes interleaved or half apart."""
    cos: torch.Tensor
    sin: torch.Tensor
    interleaved: bool

    def split(self, x):
        half = self.cos.shape[-1]
        if self.interleaved:
            return x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        return x[..., :half], x[..., half:2 * half]

    def join(self, a, b, x):
        half = self.cos.shape[-1]
        out = x.clone()
        if self.interleaved:
            out[..., 0:2 * half:2], out[..., 1:2 * half:2] = a, b
        else:
            out[..., :half], out[..., half:2 * half] = a, b
        return out

    def forth(self, x):
        a, b = self.split(x)
        return self.join(a * self.cos - b * self.sin, a * self.sin + b * self.cos, x)

    def back(self, x):
        a, b = self.split(x)
        return self.join(a * self.cos + b * self.sin, b * self.cos - a * self.sin, x)

    def size(self, x):
        """Per element the sum of the magnitudes that its rotation adds up."""
        a, b = (t.abs() for t in self.split(x))
        c, s = self.cos.abs(), self.sin.abs()
        return self.join(a * c + b * s, a * s + b * c, x.abs())


def turn_of(cos, sin, positions, axes, sections, mixed, interleaved):
    """Turn of tables [rows, half] at positions [axes, T] (None: no rotation)."""
    if cos is None:
        return None
    half = cos.shape[1]
    axis = torch.tensor(plane_axes(half, axes, sections, mixed))
    row = positions.long()[axis].t()
    plane = torch.arange(half)
    return Turn(cos.double()[row, plane][:, None], sin.double()[row, plane][:, None], interleaved)


def norm(x, w, eps):
    """(x rstd, rstd) of fp64 rows; (x, 1) without a weight."""
    if w is None:
        return x, torch.ones_like(x[..., :1])
    r = (x.square().mean(-1, keepdim=True) + eps) ** -0.5
    return x * r, r


def norm_rope(x, w, eps, turn):
    """(y, bound): fp32 arithmetic on a row keeps 2^-20 of what it adds up (a sum of d squares in a tree
    over 8 terms a lane, at most 12 roundings of 2^-24, halved by the root; rsqrtf 2^-22; five products
    and one sum more, 6 times 2^-24), then one rounding to bf16."""
    x = x.double()
    z = norm(x, w, eps)[0] * (1 if w is None else w.double())
    y, size = (z, z.abs()) if turn is None else (turn.forth(z), turn.size(z))
    return y, BF16 * y.abs() + 2.0 ** -20 * size + TINY


def norm_rope_grad(g, x, w, eps, turn):
    """((dx, bound), (dw, bound)): dx = rstd (h - n sum(n h) / d) of which every term keeps 2^-19 (the sum
    over n h, of either sign, keeps 2^-20 of its terms' magnitudes); dw sums terms that keep 2^-20 in at most
    64 roundings one after the other: 2^-18 of the terms' magnitudes."""
    g, x = g.double(), x.double()
    dz, size = (g, g.abs()) if turn is None else (turn.back(g), turn.size(g))
    if w is None:
        return (dz, BF16 * dz.abs() + 2.0 ** -20 * size + TINY), (None, None)
    n, r = norm(x, w, eps)
    w = w.double()
    h = w * dz
    dx = r * (h - n * (n * h).mean(-1, keepdim=True))
    much = r * (w.abs() * size + n.abs() * (n.abs() * w.abs() * size).mean(-1, keepdim=True))
    return ((dx, BF16 * dx.abs() + 2.0 ** -19 * much + TINY),
            ((n * dz).sum((0, 1)), 2.0 ** -18 * (n.abs() * size).sum((0, 1)) + TINY))


def within(got, want, bound, what=""):
    got = got.detach().cpu().double()
    assert torch.isfinite(got).all(), what
    err = (got - want).abs()
    assert (err <= bound).all(), (what, (err / bound).max().item())


# ---- decode behind shared prefixes ---------------------------------------------------------------

@dataclass
class SharedCase:
    q: torch.Tensor           # [T, Hq, d] bf16
    k_cache: torch.Tensor     # [P, ps, Hkv, d] bf16, every slot that no sequence holds NaN
    v_cache: torch.Tensor
    cache_seqlens: torch.Tensor
    block_table: torch.Tensor
    group_starts: torch.Tensor
    prefix_lens: torch.Tensor
    cu_seqlens_q: torch.Tensor  # None: one token a sequence
    new: list
    keys: list
    scale: float
    page_size: int
    longest: int


def shared_case(groups, Hq, Hkv, d, page_size, seed, scale=None, padding=0, decode=None, size=1.0):
    """groups: [(prefix, [(new tokens, keys behind the prefix and before them), ...]), ...].  Pages that
    a prefix fills are the group's, the one that it ends in is every sequence's own copy.  A sequence given as
    (new, None) is short: it has no more than its new tokens (of decode: 0 keys), in pages of its own."""
    gen = torch.Generator().manual_seed(seed)
    new, keys, starts, prefixes, short = [], [], [0], [], []
    for p, seqs in groups:
        for n, c in seqs:
            new.append(n)
            short.append(c is None)
            keys.append((n if decode is False or n > 1 else 0) if c is None else p + c + n)
        starts.append(len(new))
        prefixes.append(p)
    if decode is None:
        decode = all(n == 1 for n in new)
    B, ps = len(new), page_size
    lead = [p // ps for p in prefixes]
    own = []
    for g in range(len(groups)):
        for b in range(starts[g], starts[g + 1]):
            own.append(-(-keys[b] // ps) - (0 if short[b] else lead[g]))
    pages = sum(lead) + sum(own) + 2
    perm = torch.randperm(pages, generator=gen).int()
    table = torch.full((B, max([1] + [-(-k // ps) for k in keys])), -1, dtype=torch.int32)
    at = 0
    for g in range(len(groups)):
        whole = perm[at:at + lead[g]]
        at += lead[g]
        for b in range(starts[g], starts[g + 1]):
            first = 0 if short[b] else lead[g]
            table[b, :first] = whole[:first]
            table[b, first:first + own[b]] = perm[at:at + own[b]]
            at += own[b]
    caches = []
    for _ in range(2):
        x = torch.full((pages, ps, Hkv, d), math.nan)
        for g in range(len(groups)):
            lead_rows = torch.randn((prefixes[g], Hkv, d), generator=gen) * size
            for b in range(starts[g], starts[g + 1]):
                rows = torch.randn((keys[b], Hkv, d), generator=gen) * size
                if not short[b]:
                    rows[:prefixes[g]] = lead_rows
                j = torch.arange(keys[b])
                x[table[b].long()[j // ps], j % ps] = rows
        caches.append(x.to(torch.bfloat16))
    T = sum(new) + padding
    cu = None
    if not decode:
        cu = torch.tensor([0] + new).cumsum(0).int()
    else:
        assert padding == 0 and all(n == 1 for n in new)
    q = (torch.randn((T, Hq, d), generator=gen) * 1.5).to(torch.bfloat16)
    return SharedCase(q, *caches, torch.tensor(keys, dtype=torch.int32), table,
                      torch.tensor(starts, dtype=torch.int32), torch.tensor(prefixes, dtype=torch.int32),
                      cu, new, keys, d ** -0.5 if scale is None else scale, ps, max([1] + new))


def shared_exact(c):
    """(O [T, Hq, d], LSE [T, Hq], dS, W): every sequence over all its keys through its own row, with
    W = sum_j P_j |v_j| and dS = max_j scale sum_d |q_d k_jd| for the bounds."""
    T, Hq, d = c.q.shape
    Hkv = c.k_cache.shape[2]
    g = Hq // Hkv
    O, W = torch.zeros((T, Hq, d), dtype=torch.float64), torch.zeros((T, Hq, d), dtype=torch.float64)
    LSE = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    dS = torch.zeros((T, Hq), dtype=torch.float64)
    t = 0
    for b, (n, L) in enumerate(zip(c.new, c.keys)):
        if n and L:
            j = torch.arange(L)
            page = c.block_table[b].long()[j // c.page_size]
            k = c.k_cache[page, j % c.page_size].double().repeat_interleave(g, 1)
            v = c.v_cache[page, j % c.page_size].double().repeat_interleave(g, 1)
            q = c.q[t:t + n].double() * c.scale
            hidden = j > torch.arange(L - n, L)[:, None]
            x = torch.einsum("thd,khd->thk", q, k).masked_fill(hidden[:, None], -math.inf)
            lse = torch.logsumexp(x, -1)
            p = (x - torch.where(lse == -math.inf, 0.0, lse)[..., None]).exp()
            LSE[t:t + n] = lse
            O[t:t + n] = torch.einsum("thk,khd->thd", p, v)
            W[t:t + n] = torch.einsum("thk,khd->thd", p, v.abs())
            dS[t:t + n] = torch.einsum("thd,khd->thk", q.abs(), k.abs()).amax(-1)
        t += n
    return O, LSE, dS, W


def shared_check(out, lse, ref, what=""):
    """A logit is off by at most dS d 2^-23 =: x (fp32 sums of d products, each rounded in the last
    place at worst twice over), a weight therefore by the factor e^{2x}, since numerator and denominator both
    move; its rounding as a tensor-core operand is 2^-8, exp2, the sums and the merge's weights stay
    within 2^-18 together, and O is rounded to bf16: 2^-8."""
    O, LSE, dS, W = ref
    d = O.shape[-1]
    out, lse = out.detach().cpu().double(), lse.detach().cpu().double()
    empty = LSE == -math.inf
    assert torch.equal(lse == -math.inf, empty), what
    assert (out[empty] == 0).all(), what
    assert torch.isfinite(out).all(), what
    x = dS * d * 2.0 ** -23
    bound = BF16 * O.abs() + (1 + BF16) * (torch.expm1(2 * x) + BF16 + 2.0 ** -18)[..., None] * W + 1e-30
    err = (out - O).abs()
    assert (err <= bound).all(), (what, (err / bound).max().item())
    l_bound = x + 2.0 ** -20 * (2 + LSE.abs())
    l_err = (lse - LSE).abs()
    assert (l_err[~empty] <= l_bound[~empty]).all(), (what, (l_err / l_bound)[~empty].max().item())
    # the roundings are independent: on average far below the bound
    if (~empty).any():
        assert err.mean() <= 0.5 * bound.mean(), (what, (err.mean() / bound.mean()).item())
