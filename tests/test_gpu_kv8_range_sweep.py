"""Seeded random configurations of the chunk and decode calls on the 8-bit cache whose rows differ widely in
size, within a sequence and between kv heads, with single rows far above or below the others, zeros among
them; bounds as in tests.test_gpu_kv8_range."""
import random

import numpy as np
import pytest
import torch

from tests.kv8_exact import kv8_case
from tests.test_gpu_kv8 import attn  # noqa: F401
from tests.test_gpu_kv8_range import bf16, check_chunk, check_decode, put_cached

pytestmark = pytest.mark.gpu


def sizes(rng, shape):
    """Powers of two, one a row: near 2^mid per kv head, some rows up to 2^60 away, some 0."""
    mid = rng.choice([0, 0, 0, 20, -20, -50, 50], shape[1])
    e = mid + rng.uniform(-1, 1, shape) * rng.choice([1.0, 6.0, 25.0])
    far = rng.random(shape) < rng.choice([0.0, 0.01, 0.1])
    e = np.where(far, mid + rng.uniform(-60, 60, shape), e)
    return np.where(rng.random(shape) < rng.choice([0.0, 0.02]), 0.0, 2.0 ** e)


@pytest.mark.parametrize("seed", range(64))
def test_random_sizes(attn, seed):  # noqa: F811
    r = random.Random(9700 + seed)
    rng = np.random.default_rng(9700 + seed)
    Hkv, d = r.choice([1, 2, 3, 8]), r.choice([64, 128])
    g = r.choice([1, 2, 4, 7, 16])
    B = r.randint(1, 5)
    staged = r.random() < 0.6
    ctx = [r.choice([0, 1, r.randint(0, 130), r.randint(0, 700)]) for _ in range(B)]
    new = [r.choice([0, 1, r.randint(1, 9)]) for _ in range(B)]
    new[r.randrange(B)] = 1
    if staged:  # enough rows for it
        new[r.randrange(B)] = max(120, 6200 // (g * Hkv * B) + 5)
    rot = r.choice([0, 16, d // 2, d])
    causal = r.random() < 0.8
    window = r.choice([(-1, -1), (-1, -1), (r.randint(0, 200), -1), (r.randint(0, 200), r.randint(0, 40))])
    c = kv8_case(ctx, new, g * Hkv, Hkv, d, r.choice([16, 64, 192]), seed=9700 + seed, rotary_dim=rot,
                 interleaved=r.random() < 0.4)
    c.k_new = bf16(c.k_new.double().numpy() * sizes(rng, (sum(new), Hkv))[..., None])
    c.v_new = bf16(c.v_new.double().numpy() * sizes(rng, (sum(new), Hkv))[..., None])
    largest = c.k_new.double().abs().amax((0, 2)).numpy()
    for b, n in enumerate(ctx):
        if n:
            k, v = (rng.standard_normal((n, Hkv, d)) * sizes(rng, (n, Hkv))[..., None] for _ in "kv")
            put_cached(c, b, np.arange(n), k=k, v=v)
            largest = np.maximum(largest, np.abs(k).max((0, 2)))
    # queries as much smaller as the largest keys are larger: fp32 has no fractions of logits above 2^24
    size = 2.0 ** np.clip(rng.uniform(-4, 4, Hkv) - np.log2(largest + 1e-300), -100, 100)
    c.q = bf16(c.q.double().numpy() * np.repeat(size, g)[:, None])
    what = f"seed {seed}: {ctx} {new} {g}x{Hkv} d {d} rot {rot} {causal} {window}"
    check_chunk(attn, c, causal, window, what)
    c.new, c.q = [0] * B, c.q[torch.arange(B) % c.q.shape[0]].contiguous()
    check_decode(attn, c, what)
