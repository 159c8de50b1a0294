"""The 8-bit paged KV cache in fp64 numpy, written from its definition (no code of the library):
rows quantised, the cache read back, and the attention of its stored values, with the
bounds the kernels are held to.

A row x is stored as codes of the e4m3 grid and a byte b: e = the smallest integer >= -126 with
max|x| <= 448 2^e, b = e + 127, code = nearest grid value of x 2^-e (ties to the even code).
"""
import dataclasses

import numpy as np
import torch

from exact_attention_70_gb300 import synth
from oracle import oracle

# the 127 non-negative finite values by code: subnormals in steps of 2^-9, then 8..15 / 8 times 2^k
GRID = np.array([c * 2.0 ** -9 if c < 8 else (8 + c % 8) * 2.0 ** (c // 8 - 10)
                 for c in range(127)])
NAN_CODE = 0x7F
VALUES = np.concatenate([GRID, [np.nan], -GRID, [np.nan]])


def quantise_rows(x):
    """fp64 rows [..., d] -> (uint8 codes [..., d], uint8 scale bytes [...])."""
    x = np.asarray(x, np.float64)
    finite = np.isfinite(x)
    top = np.where(finite, np.abs(x), 0.0).max(axis=-1)
    m, ex = np.frexp(top)  # top = m 2^ex with m in [0.5, 1); 448 = 0.875 2^9
    e = np.where(top > 0, np.maximum(ex - 9 + (m > 0.875), -126), -126)
    y = np.abs(np.where(finite, x, 0.0)) * np.exp2(-e.astype(np.float64))[..., None]
    hi = np.clip(np.searchsorted(GRID, y), 1, 126)
    up, down = GRID[hi] - y, y - GRID[hi - 1]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)
    code = np.where(np.signbit(x), code + 128, code)
    return np.where(finite, code, NAN_CODE).astype(np.uint8), (e + 127).astype(np.uint8)


def rotate(x, pos, cos, sin, interleaved):
    """fp64 rows x [n, H, d] at positions pos [n]; tables fp32 [rows, rot / 2] (or None)."""
    x = np.array(x, np.float64)
    if cos is None:
        return x
    c = cos.numpy().astype(np.float64)[pos][:, None]
    s = sin.numpy().astype(np.float64)[pos][:, None]
    half = c.shape[-1]
    a, b = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved
            else (slice(0, half), slice(half, 2 * half)))
    xa, xb = x[..., a].copy(), x[..., b].copy()
    x[..., a], x[..., b] = xa * c - xb * s, xa * s + xb * c
    return x


@dataclasses.dataclass
class Kv8Case:
    """New tokens q_lens over ctx_lens cached ones (q_lens None: decode, ctx_lens are all keys)."""
    q: torch.Tensor
    k_new: torch.Tensor
    v_new: torch.Tensor
    k_cache: torch.Tensor
    v_cache: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor
    cache_seqlens: torch.Tensor
    block_table: torch.Tensor
    cu_seqlens_q: torch.Tensor
    rotary_cos: torch.Tensor
    rotary_sin: torch.Tensor
    ctx: list
    new: list
    page_size: int
    interleaved: bool
    scale: float

    @property
    def cache(self):
        return self.k_cache, self.v_cache, self.k_scale, self.v_scale


def kv8_case(ctx_lens, q_lens, Hq, Hkv, d, page_size, seed, rotary_dim=0, interleaved=False,
             spread=2.0, scale=None, padding=0, spare_pages=2):
    """Cached rows are quantised N(0, 1) rows times 2^U(-spread, spread); every slot that holds no
    cached token gets the NaN code and the NaN scale byte, every table entry that no token
    needs is -1, and `padding` rows follow the last sequence's."""
    rng = np.random.default_rng(seed)
    decode = q_lens is None
    new = [0] * len(ctx_lens) if decode else list(q_lens)
    lens = [c + n for c, n in zip(ctx_lens, new)]
    per = [(n + page_size - 1) // page_size for n in lens]
    P = sum(per) + spare_pages
    perm = rng.permutation(P)
    table = np.full((len(lens), max([1] + per)), -1, np.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = perm[at:at + n]
        at += n
    caches = []
    for _ in range(2):
        codes = np.full((P, page_size, Hkv, d), NAN_CODE, np.uint8)
        bytes_ = np.full((P, Hkv, page_size), 255, np.uint8)
        for b, c in enumerate(ctx_lens):
            x = rng.standard_normal((c, Hkv, d)) * 2.0 ** rng.uniform(-spread, spread, (c, Hkv, 1))
            qc, qb = quantise_rows(x)
            j = np.arange(c)
            codes[table[b, j // page_size], j % page_size] = qc
            bytes_[table[b, j // page_size], :, j % page_size] = qb
        caches += [torch.from_numpy(codes), torch.from_numpy(bytes_)]
    T = (len(lens) if decode else sum(new)) + padding
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(torch.bfloat16)  # noqa: E731
    cos = sin = None
    if rotary_dim:
        cos, sin = synth.rotary_tables(max(lens) + 1, rotary_dim)
    return Kv8Case(q=bf(T, Hq, d), k_new=bf(T, Hkv, d), v_new=bf(T, Hkv, d), k_cache=caches[0],
                   v_cache=caches[2], k_scale=caches[1], v_scale=caches[3],
                   cache_seqlens=torch.tensor(ctx_lens, dtype=torch.int32),
                   block_table=torch.from_numpy(table), cu_seqlens_q=synth.cu_from_lengths(new),
                   rotary_cos=cos, rotary_sin=sin, ctx=list(ctx_lens), new=new,
                   page_size=page_size, interleaved=interleaved,
                   scale=d ** -0.5 if scale is None else scale)


def appended(c):
    """The four cache arrays (numpy) after the append of c's new tokens."""
    out = [t.numpy().copy() for t in c.cache]
    t0 = 0
    for b, n in enumerate(c.new):
        if n:
            pos = c.ctx[b] + np.arange(n)
            page, slot = c.block_table.numpy()[b, pos // c.page_size], pos % c.page_size
            k = rotate(c.k_new[t0:t0 + n].double().numpy(), pos, c.rotary_cos, c.rotary_sin,
                       c.interleaved)
            for i, x in ((0, k), (1, c.v_new[t0:t0 + n].double().numpy())):
                codes, sb = quantise_rows(x)
                out[i][page, slot] = codes
                out[i + 2][page, :, slot] = sb
        t0 += n
    return out


def read_back(arrays, table, b, n, page_size):
    """fp64 (k, v) [n, Hkv, d] of sequence b's first n tokens."""
    j = np.arange(n)
    page, slot = table[b, j // page_size], j % page_size
    return [VALUES[arrays[i][page, slot]]
            * np.exp2(arrays[i + 2][page, :, slot].astype(np.float64) - 127.0)[..., None]
            for i in (0, 1)]


def attention(c, arrays, causal=True, window=(-1, -1)):
    """(O [T, Hq, d], LSE [T, Hq], dS, W): the oracle's attention of the stored values and the
    exactly rotated queries over c's tokens, and per element W = sum_j P_j |v_j| and per row
    dS = max_j scale sum_d |q_d k_jd| for the error bounds."""
    decode = not any(c.new)
    table = c.block_table.numpy()
    T, Hq, d = c.q.shape
    Hkv = c.k_cache.shape[2]
    O, LSE = np.zeros((T, Hq, d)), np.full((T, Hq), -np.inf)
    dS, W = np.zeros((T, Hq)), np.zeros((T, Hq, d))
    t0 = 0
    for b in range(len(c.ctx)):
        n, L = (1, c.ctx[b]) if decode else (c.new[b], c.ctx[b] + c.new[b])
        if n == 0:
            continue
        q = c.q[t0:t0 + n].double().numpy()
        if not decode:
            q = rotate(q, c.ctx[b] + np.arange(n), c.rotary_cos, c.rotary_sin, c.interleaved)
        k, v = read_back(arrays, table, b, L, c.page_size)
        cu = np.array([0, n], np.int32), np.array([0, L], np.int32)
        o, lse = oracle.attn_fwd(q, k, v, *cu, c.scale, causal, *window)
        w, _ = oracle.attn_fwd(q, k, np.abs(v), *cu, c.scale, causal, *window)
        O[t0:t0 + n], LSE[t0:t0 + n], W[t0:t0 + n] = o, lse.T, w
        if L:
            for h in range(Hq):
                dS[t0:t0 + n, h] = c.scale * (np.abs(q[:, h]) @ np.abs(k[:, h // (Hq // Hkv)]).T).max(1)
        t0 += n
    return O, LSE, dS, W


def check(out, lse, ref, u_p, rotated, what=""):
    """The kernels' O (bf16) and LSE against `attention`'s, within what their roundings allow.

    A logit is off by at most dS times (d 2^-23: the fp32 sums of d products, each rounded in the
    last place at worst twice over, plus 2^-8 where the query was rounded to bf16 after its
    rotation) =: x; a weight therefore by the factor e^{2x}, since numerator and denominator
    both move; its rounding as a tensor-core operand is u_p (2^-11 f16, 2^-8 bf16) and exp2 and the
    division stay within 2^-20 together.  O is rounded to bf16: 2^-8."""
    O, LSE, dS, W = ref
    d = O.shape[-1]
    out = out.double().cpu().numpy()
    lse = lse.double().cpu().numpy()
    empty = ~np.isfinite(LSE)
    assert np.array_equal(np.isneginf(lse), empty), what
    assert np.all(out[empty] == 0.0), what
    x = dS * (d * 2.0 ** -23 + (2.0 ** -20 if rotated else 0.0))
    p_err = np.expm1(2 * x) + u_p + 2.0 ** -20
    bound = 2.0 ** -8 * np.abs(O) + (1 + 2.0 ** -8) * p_err[..., None] * W
    err = np.abs(out - O)
    assert np.all(np.isfinite(out)), what
    assert np.all(err <= bound + 1e-30), (what, (err / np.maximum(bound, 1e-30)).max())
    l_err = np.abs(lse[~empty] - LSE[~empty])
    l_bound = (x + 2.0 ** -20 * (2 + np.abs(np.where(empty, 0, LSE))))[~empty]
    assert np.all(l_err <= l_bound), (what, (l_err / l_bound).max())
    # the roundings are independent: on average far below the bound
    if err.size:
        assert err.mean() <= 0.5 * bound.mean() + 1e-30, (what, err.mean() / bound.mean())
