"""The calls on the 8-bit paged KV cache over the whole range of what it stores and of what a mask
leaves out, against the fp64 definition (tests.kv8_exact): rows of zeros, keys and values from
2^-126 to 2^127, values far apart within a sequence, large, infinite and NaN values that no row sees,
pages that a window has left behind.

The bounds are those of kv8_exact.check: a logit is off by dS d 2^-23 for its fp32 sums of d products
(and dS 2^-20 where the query was rotated and goes to the tensor cores as two f16 numbers of 11 bits
each), a weight by 2^-11 as an f16 operand and by 2^-20 for exp2 and the division, O by 2^-8 as
bf16."""
import numpy as np
import pytest
import torch

from tests import kv8_exact
from tests.kv8_exact import kv8_case
from tests.test_gpu_kv8 import append, attn, gpu_cache  # noqa: F401

pytestmark = pytest.mark.gpu



def bf16(x):
    return torch.as_tensor(x).to(torch.bfloat16)


def put_cached(c, b, j, k=None, v=None):
    """Stores fp64 rows k, v [n, Hkv, d] as cached tokens j [n] of sequence b."""
    j = np.asarray(j)
    page = torch.from_numpy(c.block_table.numpy()[b, j // c.page_size].astype(np.int64))
    slot = torch.from_numpy(j % c.page_size)
    for x, codes, scale in ((k, c.k_cache, c.k_scale), (v, c.v_cache, c.v_scale)):
        if x is not None:
            q, s = kv8_exact.quantise_rows(x)
            codes[page, slot], scale[page, :, slot] = torch.from_numpy(q), torch.from_numpy(s)


def new_rows(c, b):
    """The rows of sequence b's new tokens."""
    cu = c.cu_seqlens_q.tolist()
    return slice(cu[b], cu[b + 1])


@pytest.mark.parametrize("rotary,inter", [(64, False), (32, True), (48, False)])
@pytest.mark.parametrize("e", [-133, -130, -128, -126, -122, -118, -100, 0, 100, 120, 126, 127])
def test_append_rotates_rows_of_any_size(attn, e, rotary, inter):  # noqa: F811
    """Exact bytes for rows of size 2^e: with low parts of the products below fp32's range, and with
    rotated elements above it."""
    c = kv8_case([11, 0], [700, 300], 2, 2, 64, 32, seed=450, rotary_dim=rotary, interleaved=inter)
    top = float(torch.finfo(torch.bfloat16).max)
    c.k_new = bf16(np.clip(c.k_new.double().numpy() * 2.0 ** e, -top, top))
    c.k_new[5, 0] = bf16([top, -top] * 32)
    c.k_new[6, 0], c.k_new[7, 1] = 0, -0.0
    c.k_new[8, 0, 3], c.k_new[9, 1, 40], c.k_new[10, 1, 2] = float("nan"), float("inf"), -float("inf")
    cache = gpu_cache(c)
    append(attn, c, cache)
    assert attn.attn_get_device_status() == 0
    # a pair with an element that is not finite: both of its rotated elements are not
    rows = np.isfinite(c.k_new.float().numpy()).all(-1)
    arrays = kv8_exact.appended(c)
    got = [t.cpu().numpy() for t in cache]
    for i in (1, 3):
        assert np.array_equal(got[i], arrays[i])
    t = np.arange(1000)
    b = (t >= 700).astype(int)
    pos = np.where(b == 0, 11 + t, t - 700)
    page, slot = c.block_table.numpy()[b, pos // 32], pos % 32
    # (an exact 0, the sum of two zeros, has no sign: either code of it will do)
    exact = np.concatenate([kv8_exact.rotate(c.k_new[new_rows(c, i)].double().numpy(), pos[b == i], c.rotary_cos,
                                             c.rotary_sin, inter) for i in (0, 1)])
    codes = [np.where((exact == 0) & (x[page, slot] == 0x80), 0, x[page, slot]) for x in (got[0], arrays[0])]
    assert np.array_equal(codes[0][rows], codes[1][rows])
    assert np.array_equal(got[2][page, :, slot][rows], arrays[2][page, :, slot][rows])
    for x, y in ((got[0], arrays[0]), (got[2], arrays[2])):   # and nothing else was written
        for z in (x, y):
            z[(page, slot) if z.ndim == 4 else (page, slice(None), slot)] = 0
        assert np.array_equal(x, y)
