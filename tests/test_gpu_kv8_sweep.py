"""Seeded random configurations of the calls on the 8-bit paged KV cache against its fp64
definition: head pairings, page sizes, rotations, windows and lengths (empty sequences and
single tokens among them), with every unused slot and table entry poisoned."""
import random

import numpy as np
import pytest
import torch

from tests import kv8_exact
from tests.kv8_exact import kv8_case
from tests.test_gpu_kv8 import append, attn, chunk, decode, dev, gpu_cache, same_cache  # noqa: F401

pytestmark = pytest.mark.gpu


def draw(seed):
    r = random.Random(9000 + seed)
    Hkv = r.choice([1, 2, 3, 8])
    g = r.choice([1, 2, 3, 4, 7, 16, 20])
    d = r.choice([64, 128])
    ps = r.choice([16, 32, 64, 128, 192, 256])
    B = r.randint(1, 6)
    ctx = [r.choice([0, 1, r.randint(0, 130), r.randint(0, 1500)]) for _ in range(B)]
    most = max(1, 3000 // (g * Hkv))
    new = [r.choice([0, 1, r.randint(1, 9), r.randint(1, min(700, most))]) for _ in range(B)]
    if not any(new):
        new[0] = 1
    rot = r.choice([0, 16, d // 2, d, d - 16])
    causal = r.random() < 0.8
    window = r.choice([(-1, -1), (-1, -1), (r.randint(0, 300), -1), (r.randint(0, 300), r.randint(0, 40))])
    return r, dict(ctx_lens=ctx, q_lens=new, Hq=g * Hkv, Hkv=Hkv, d=d, page_size=ps, rotary_dim=rot,
                   interleaved=r.random() < 0.4), causal, window


@pytest.mark.parametrize("seed", range(48))
def test_random_configuration(attn, seed):  # noqa: F811
    r, k, causal, window = draw(seed)
    what = f"seed {seed}: {k} {causal} {window}"
    c = kv8_case(**k, seed=9500 + seed, spread=0.5, padding=r.choice([0, 2]))
    T = sum(c.new)
    arrays = kv8_exact.appended(c)
    cache = gpu_cache(c)
    append(attn, c, cache)
    same_cache(cache, arrays)
    cache = gpu_cache(c)
    out, lse = chunk(attn, c, cache, causal, window,
                     max_total_k=r.choice([None, sum(c.ctx) + T + 1000]))
    assert attn.attn_get_device_status() == 0, what
    same_cache(cache, arrays)
    ref = [x[:T] for x in kv8_exact.attention(c, arrays, causal, window)]
    kv8_exact.check(out[:T], lse[:, :T].t(), ref, 2.0 ** -11, c.rotary_cos is not None, what)
    # then one token a sequence over what is cached now, and the cache read back
    c.ctx, c.new = [a + b for a, b in zip(c.ctx, c.new)], [0] * len(c.ctx)
    c.cache_seqlens = torch.tensor(c.ctx, dtype=torch.int32)
    g = torch.Generator().manual_seed(seed)
    c.q = torch.randn(len(c.ctx), k["Hq"], k["d"], generator=g).to(torch.bfloat16)
    out, lse = decode(attn, c, cache)
    kv8_exact.check(out, lse, kv8_exact.attention(c, arrays), 2.0 ** -11, False, what)
    cu = np.concatenate([[0], np.cumsum(c.ctx)]).astype(np.int32)
    kk, vv = attn.attn_kvcache_read_fp8(*cache, dev(c.block_table), torch.from_numpy(cu).cuda(), int(cu[-1]))
    assert attn.attn_get_device_status() == 0, what
    for b, n in enumerate(c.ctx):
        k_ref, v_ref = kv8_exact.read_back(arrays, c.block_table.numpy(), b, n, c.page_size)
        assert np.array_equal(kk[cu[b]:cu[b + 1]].double().cpu().numpy(), k_ref), what
        assert np.array_equal(vv[cu[b]:cu[b + 1]].double().cpu().numpy(), v_ref), what
