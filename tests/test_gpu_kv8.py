"""The 8-bit paged KV cache on the GPU against its fp64 definition (tests.kv8_exact): the
written bytes and the values read back bit for bit, decode and chunk attention within the bounds
their roundings allow.  Every slot that holds no token carries the NaN code and the NaN scale
byte, and every table entry that no token needs is -1."""
import numpy as np
import pytest
import torch

from tests import kv8_exact
from tests.kv8_exact import kv8_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def attn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from exact_attention_70_gb300 import build as attn_build
    attn_build.build()
    from exact_attention_70_gb300 import binding
    binding.load()
    return binding


def dev(t):
    return None if t is None else t.cuda()


def gpu_cache(c):
    return [t.cuda() for t in c.cache]


def append(attn, c, cache):
    attn.attn_kvcache_append_fp8(dev(c.k_new), dev(c.v_new), *cache, dev(c.cache_seqlens),
                                 dev(c.block_table), dev(c.cu_seqlens_q), dev(c.rotary_cos),
                                 dev(c.rotary_sin), c.interleaved)


def decode(attn, c, cache=None, **kw):
    out, lse = attn.attn_decode_kvcache_fp8(dev(c.q), *(cache or gpu_cache(c)),
                                            dev(c.cache_seqlens), dev(c.block_table), c.scale, **kw)
    torch.cuda.synchronize()
    assert attn.attn_get_device_status() == 0
    return out, lse


def chunk(attn, c, cache, causal=True, window=(-1, -1), max_total_k=None, **kw):
    out, lse = attn.attn_fwd_kvcache_fp8(
        dev(c.q), dev(c.k_new), dev(c.v_new), *cache, dev(c.cache_seqlens), dev(c.block_table),
        dev(c.cu_seqlens_q), max(c.new),
        sum(c.ctx) + sum(c.new) if max_total_k is None else max_total_k, c.scale, causal, *window,
        dev(c.rotary_cos), dev(c.rotary_sin), c.interleaved, **kw)
    torch.cuda.synchronize()
    return out, lse


def same_cache(cache, arrays):
    for got, want in zip(cache, arrays):
        assert np.array_equal(got.cpu().numpy(), want)


APPEND = [
    # ctx, q, Hkv, d, page, rotary, interleaved
    ([0], [1], 1, 64, 16, 0, False),
    ([5, 0, 63, 700], [1, 1, 1, 1], 8, 128, 256, 128, False),
    ([0, 17, 900, 3], [130, 0, 257, 1], 3, 64, 16, 32, True),
    ([64, 1], [200, 63], 2, 128, 64, 128, True),
    ([100, 40], [33, 500], 5, 128, 32, 48, False),
    ([9, 0, 0], [0, 0, 77], 4, 64, 128, 64, False),
]


@pytest.mark.parametrize("i", range(len(APPEND)))
@pytest.mark.parametrize("padding", [0, 7])
def test_append_writes_the_exact_bytes(attn, i, padding):
    ctx, q, Hkv, d, ps, rot, inter = APPEND[i]
    c = kv8_case(ctx, q, Hkv, Hkv, d, ps, seed=20 + i, rotary_dim=rot, interleaved=inter,
                 padding=padding)
    cache = gpu_cache(c)
    append(attn, c, cache)
    assert attn.attn_get_device_status() == 0
    same_cache(cache, kv8_exact.appended(c))  # the tokens' slots and nothing else


def test_append_extreme_rows(attn):
    c = kv8_case([0], [12], 1, 1, 64, 16, seed=30)
    x = torch.zeros(12, 1, 64)
    g = torch.Generator().manual_seed(30)
    r = torch.randn(64, generator=g)
    x[1, 0] = r * 1e38
    x[2, 0] = r * 1e-38           # below the smallest scale's normal codes
    x[3, 0] = r * 2.0 ** -133     # bf16 subnormals
    x[4, 0] = r
    x[4, 0, 3] = float("nan")
    x[5, 0] = r
    x[5, 0, 7], x[5, 0, 63] = float("inf"), float("-inf")
    x[6, 0] = float("inf")
    x[7, 0, 0] = 448.0            # on the border of a scale
    x[8, 0, 0] = 450.0            # just above it
    x[9, 0] = -0.0
    x[10, 0] = torch.tensor([1.0, 1.0625, 1.1875, 1.4375] * 16)  # ties
    x[11, 0, 63] = 3.3895e38
    c.k_new, c.v_new = x.to(torch.bfloat16), x.flip(0).contiguous().to(torch.bfloat16)
    cache = gpu_cache(c)
    append(attn, c, cache)
    assert attn.attn_get_device_status() == 0
    same_cache(cache, kv8_exact.appended(c))


@pytest.mark.parametrize("i", range(6))
def test_read_returns_the_stored_values(attn, i):
    lens, Hkv, d, ps = [([1], 1, 64, 16), ([0, 5, 0], 2, 128, 64), ([300, 0, 77, 1000], 8, 128, 256),
                        ([129, 15, 16, 17], 3, 64, 16), ([500], 5, 128, 32), ([64, 640], 4, 64, 128)][i]
    c = kv8_case(lens, None, Hkv, Hkv, d, ps, seed=40 + i, spread=20.0)
    T = sum(lens)
    cu = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).cuda()
    k = torch.full((T + 5, Hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    v = torch.full_like(k, -7.0)
    attn.attn_kvcache_read_fp8(*gpu_cache(c), dev(c.block_table), cu, T + 5, k=k, v=v)
    assert attn.attn_get_device_status() == 0
    arrays = [t.numpy() for t in c.cache]
    rows = [kv8_exact.read_back(arrays, c.block_table.numpy(), b, n, ps) for b, n in enumerate(lens)]
    for got, fill, j in ((k, 7.0, 0), (v, -7.0, 1)):
        assert np.array_equal(got[:T].double().cpu().numpy(), np.concatenate([r[j] for r in rows]))
        assert (got[T:] == fill).all()  # rows behind the last sequence are left as they were


def test_read_special_codes_and_scales(attn):
    """All 256 codes under the smallest, a middle, a large and the NaN scale."""
    codes = torch.arange(256, dtype=torch.uint8).view(1, 1, 4, 64).repeat(1, 16, 1, 1).contiguous()
    scale = torch.full((1, 4, 16), 255, dtype=torch.uint8)
    for j, b in enumerate([1, 100, 127, 200, 240, 0]):
        scale[:, :, j] = b
    cu = torch.tensor([0, 7], dtype=torch.int32)
    k, v = attn.attn_kvcache_read_fp8(codes.cuda(), codes.cuda(), scale.cuda(), scale.cuda(),
                                      torch.zeros((1, 1), dtype=torch.int32).cuda(), cu.cuda(), 7)
    want = kv8_exact.VALUES.reshape(1, 4, 64) * np.exp2(
        np.array([1, 100, 127, 200, 240, 0, np.nan]) - 127)[:, None, None]
    want = torch.from_numpy(want).to(torch.bfloat16)  # (subnormal results round)
    for got in (k, v):
        assert torch.equal(torch.nan_to_num(got.cpu(), nan=9.0), torch.nan_to_num(want, nan=9.0))


DECODE = [
    # lengths, Hq, Hkv, d, page
    ([1], 1, 1, 64, 16),
    ([0, 1, 2, 63, 64, 65], 8, 2, 128, 64),
    ([700], 8, 2, 64, 64),
    ([5, 700, 0, 2000, 333], 14, 2, 128, 16),
    ([1000, 4097], 32, 8, 128, 256),
    ([300, 20], 16, 1, 64, 32),
    ([77, 513], 40, 1, 128, 128),   # more heads than one CTA's rows
    ([2500], 12, 4, 64, 128),
    ([40 * i % 997 for i in range(100)], 4, 2, 64, 16),     # more sequences than a warp has lanes
    ([9000, 1, 0, 20000], 8, 4, 128, 192),                  # units cut into many parts
    ([100000], 2, 1, 64, 64),
    ([128 * (i % 3) for i in range(700)], 2, 1, 64, 64),    # many units a CTA, whole and cut
    ([300, 9], 200, 1, 64, 16),                             # a group of 200 heads
    ([50, 3], 400, 400, 64, 16),                            # more kv heads than CTAs
]


@pytest.mark.parametrize("i", range(len(DECODE)))
def test_decode_matches_the_definition(attn, i):
    lens, Hq, Hkv, d, ps = DECODE[i]
    c = kv8_case(lens, None, Hq, Hkv, d, ps, seed=50 + i)
    out, lse = decode(attn, c)
    ref = kv8_exact.attention(c, [t.numpy() for t in c.cache])
    kv8_exact.check(out, lse, ref, 2.0 ** -11, False, f"decode{i}")


def test_decode_with_tiny_and_large_rows(attn):
    """Queries and cached rows of very different magnitudes: row scales stay outside the products."""
    c = kv8_case([300, 40], None, 8, 2, 128, 64, seed=70, spread=6.0, scale=1e-3)
    c.q = (c.q.float() * torch.tensor([1e-20, 30.0, 1e-3, 1.0, 0.0, 8.0, 1e-38, 2.0])[:, None]).to(torch.bfloat16)
    out, lse = decode(attn, c)
    kv8_exact.check(out, lse, kv8_exact.attention(c, [t.numpy() for t in c.cache]), 2.0 ** -11, False)


def test_decode_zero_values_beside_large_ones(attn):
    """An all-zero row has the smallest scale: it must not disturb its neighbours' precision."""
    c = kv8_case([100], None, 4, 1, 64, 16, seed=71)
    codes, sb = kv8_exact.quantise_rows(np.zeros((1, 64)))
    page = int(c.block_table[0, 2])
    for t, s in ((c.v_cache, c.v_scale), (c.k_cache, c.k_scale)):
        t[page, 3:9, 0], s[page, 0, 3:9] = torch.from_numpy(codes), int(sb[0])
    out, lse = decode(attn, c)
    kv8_exact.check(out, lse, kv8_exact.attention(c, [t.numpy() for t in c.cache]), 2.0 ** -11, False)


CHUNK = [
    # ctx, q, Hq, Hkv, d, page, rotary, interleaved, causal, window
    ([8, 11, 5], [4, 1, 1], 4, 2, 128, 16, 0, False, True, (-1, -1)),
    ([0, 500, 1000], [300, 77, 1], 8, 2, 128, 64, 128, False, True, (-1, -1)),
    ([1000, 33], [129, 256], 32, 8, 128, 256, 64, False, True, (-1, -1)),
    ([3000], [200], 4, 4, 64, 128, 64, True, True, (300, 0)),
    ([127, 128, 129, 0, 9], [1, 2, 3, 130, 0], 16, 1, 128, 32, 32, False, True, (-1, -1)),
    ([0], [500], 4, 2, 128, 16, 0, False, False, (-1, -1)),
    ([640, 7], [64, 200], 8, 8, 64, 16, 16, True, True, (100, 0)),
    ([50, 300], [40, 5], 6, 2, 64, 64, 0, False, False, (30, 7)),   # both sides bounded
    ([2000], [4], 8, 2, 128, 64, 128, False, True, (0, 0)),         # a row sees itself alone
    ([1500, 10], [3, 9], 20, 1, 128, 128, 64, False, True, (-1, -1)),
    ([0, 0, 700, 5], [0, 129, 1, 300], 4, 4, 128, 16, 128, True, True, (64, -1)),
    ([300, 77], [50, 140], 12, 4, 64, 192, 0, False, False, (-1, 20)),
    # enough rows for the staged path
    ([3000, 40], [200, 90], 32, 8, 64, 128, 64, True, True, (300, 0)),
    ([0], [250], 32, 8, 128, 16, 0, False, False, (-1, -1)),
    ([640, 7, 0, 3], [64, 200, 1, 0], 64, 8, 64, 16, 16, True, True, (100, 0)),
    ([50, 300, 900], [40, 90, 2], 30, 10, 64, 64, 0, False, False, (30, 7)),
    ([700, 5], [1, 100], 128, 2, 128, 192, 128, False, True, (64, -1)),
    ([0, 130], [400, 300], 16, 8, 128, 32, 96, False, True, (-1, -1)),
    ([5], [40], 160, 1, 64, 16, 64, False, True, (-1, -1)),   # more heads a group than a tile packs
]


@pytest.mark.parametrize("padding", [0, 3])
@pytest.mark.parametrize("i", range(len(CHUNK)))
def test_chunk_matches_the_definition(attn, i, padding):
    ctx, q, Hq, Hkv, d, ps, rot, inter, causal, window = CHUNK[i]
    c = kv8_case(ctx, q, Hq, Hkv, d, ps, seed=80 + i, rotary_dim=rot, interleaved=inter,
                 spread=0.5, padding=padding)
    cache = gpu_cache(c)
    out = torch.full((sum(q) + padding, Hq, d), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((Hq, sum(q) + padding), 3.0, device="cuda")
    chunk(attn, c, cache, causal, window, out=out, lse=lse)
    assert attn.attn_get_device_status() == 0
    arrays = kv8_exact.appended(c)
    same_cache(cache, arrays)
    T = sum(q)
    ref = [x[:T] for x in kv8_exact.attention(c, arrays, causal, window)]
    kv8_exact.check(out[:T], lse[:, :T].t(), ref, 2.0 ** -11, rot > 0, f"chunk{i}")
    assert (out[T:] == 3.0).all() and (lse[:, T:] == 3.0).all()


def test_a_generation_from_prompt_to_tokens(attn):
    """The calls as a server makes them: a prompt in two chunks, then single tokens, each step's
    cache and output against the definition; at the end the cache read back and attended to by
    attn_fwd."""
    Hq, Hkv, d, ps = 8, 2, 128, 16
    total = kv8_case([0, 0], [96, 61], Hq, Hkv, d, ps, seed=110, rotary_dim=128, spread=0.0)
    cache = gpu_cache(total)
    arrays = [t.numpy().copy() for t in total.cache]
    cu = total.cu_seqlens_q.tolist()
    done = [0, 0]
    for step in ([40, 0], [50, 58], [1, 1], [1, 1], [4, 1]):
        pick = torch.cat([torch.arange(cu[b] + done[b], cu[b] + done[b] + step[b]) for b in (0, 1)])
        c = kv8_case(done, step, Hq, Hkv, d, ps, seed=111, rotary_dim=128)
        c.q, c.k_new, c.v_new = total.q[pick], total.k_new[pick], total.v_new[pick]
        c.block_table, c.rotary_cos, c.rotary_sin = total.block_table, total.rotary_cos, total.rotary_sin
        c.k_cache, c.v_cache, c.k_scale, c.v_scale = (torch.from_numpy(a) for a in arrays)
        arrays = kv8_exact.appended(c)
        ref = kv8_exact.attention(c, arrays)
        if step == [1, 1]:
            # append and decode as calls of their own (no rotation of q in the decode call)
            append(attn, c, cache)
            c.q = torch.from_numpy(np.stack([
                kv8_exact.rotate(c.q[b:b + 1].double().numpy(), np.array([done[b]]), c.rotary_cos,
                                 c.rotary_sin, False)[0] for b in (0, 1)])).to(torch.bfloat16)
            c.ctx, c.new = [n + 1 for n in done], [0, 0]
            c.cache_seqlens = torch.tensor(c.ctx, dtype=torch.int32)
            out, lse = decode(attn, c, cache)
            ref = kv8_exact.attention(c, arrays)
            kv8_exact.check(out, lse, ref, 2.0 ** -11, False, "step")
        else:
            out, lse = chunk(attn, c, cache)
            kv8_exact.check(out, lse.t(), ref, 2.0 ** -11, True, "chunk")
        same_cache(cache, arrays)
        done = [a + b for a, b in zip(done, step)]
    assert attn.attn_get_device_status() == 0
    cu_k = torch.tensor([0, done[0], sum(done)], dtype=torch.int32)
    k, v = attn.attn_kvcache_read_fp8(*cache, dev(total.block_table), cu_k.cuda(), sum(done))
    out, lse = attn.attn_fwd(dev(total.q), k, v, dev(total.cu_seqlens_q), cu_k.cuda(), 96, 96,
                             causal=True)
    c = kv8_case([0, 0], done, Hq, Hkv, d, ps, seed=112)
    c.q, c.block_table, c.rotary_cos = total.q, total.block_table, None
    kv8_exact.check(out, lse.t(), kv8_exact.attention(c, arrays), 2.0 ** -8, False, "attn_fwd")


@pytest.mark.parametrize("q", [3, 200])
def test_chunk_with_rows_of_very_different_scales(attn, q):
    """Cached and new rows 2^24 apart, in both ways a chunk is computed."""
    c = kv8_case([100, 257], [q, q // 2], 32, 8, 64, 32, seed=115, rotary_dim=64, spread=6.0, scale=2e-3)
    f = 2.0 ** torch.arange(-6, 7).float().repeat(q)[:c.k_new.shape[0], None, None]
    c.k_new, c.v_new = (c.k_new.float() * f).to(torch.bfloat16), (c.v_new.float() / f).to(torch.bfloat16)
    cache = gpu_cache(c)
    out, lse = chunk(attn, c, cache)
    assert attn.attn_get_device_status() == 0
    arrays = kv8_exact.appended(c)
    same_cache(cache, arrays)
    kv8_exact.check(out, lse.t(), kv8_exact.attention(c, arrays), 2.0 ** -11, True)


def test_nan_in_a_visible_token_reaches_its_rows_only(attn):
    c = kv8_case([40, 50], None, 4, 2, 64, 16, seed=120)
    c.k_cache[int(c.block_table[1, 1]), 3, 0, 5] = 0x7F   # kv head 0 of sequence 1
    out, lse = decode(attn, c)
    assert torch.isnan(out[1, :2]).all() and torch.isnan(lse[1, :2]).all()
    ref = kv8_exact.attention(c, [t.numpy() for t in c.cache])
    keep = ((0, slice(None)), (1, slice(2, 4)))
    for b, h in keep:
        kv8_exact.check(out[b:b + 1, h], lse[b:b + 1, h], [x[b:b + 1, h] for x in ref], 2.0 ** -11, False)


def test_bad_pages_and_lengths_are_reported(attn):
    def status():
        s = attn.attn_get_device_status()
        assert attn.attn_get_device_status() == 0
        return s

    c = kv8_case([100, 30], [20, 3], 4, 2, 64, 16, seed=130)
    for bad in (10 ** 6, -5):
        c.block_table[0, 6] = bad          # positions 96-111: cached and new tokens
        cache = gpu_cache(c)
        append(attn, c, cache)
        assert status() == -6
        chunk(attn, c, cache)
        assert status() == -6
        cu = torch.tensor([0, 110, 140], dtype=torch.int32).cuda()
        attn.attn_kvcache_read_fp8(*cache, dev(c.block_table), cu, 140)
        assert status() == -6
        attn.attn_decode_kvcache_fp8(dev(c.q[:2]), *cache, dev(c.cache_seqlens), dev(c.block_table))
        assert status() == -6
    c = kv8_case([100, 30], [20, 3], 4, 2, 64, 16, seed=131, rotary_dim=64)
    for lens in ([-1, 30], [10 ** 6, 30], [2 ** 31 - 1, 30]):
        c.cache_seqlens = torch.tensor(lens, dtype=torch.int32)
        cache = gpu_cache(c)
        append(attn, c, cache)
        assert status() == -6
        chunk(attn, c, cache)
        assert status() == -6
        attn.attn_decode_kvcache_fp8(dev(c.q[:2]), *cache, dev(c.cache_seqlens), dev(c.block_table))
        assert status() == -6
    c = kv8_case([100, 30], [20, 3], 4, 2, 64, 16, seed=132, rotary_dim=64)
    c.rotary_cos, c.rotary_sin = c.rotary_cos[:110], c.rotary_sin[:110]   # tables too short
    append(attn, c, gpu_cache(c))
    assert status() == -6
    c = kv8_case([100, 30], [20, 3], 4, 2, 64, 16, seed=133)
    c.new = [19, 3]                                                       # max_seqlen_q too small
    chunk(attn, c, gpu_cache(c), max_total_k=153)
    assert status() == -6
    c = kv8_case([900, 30], [100, 3], 32, 8, 64, 16, seed=133)
    chunk(attn, c, gpu_cache(c), max_total_k=700)                         # max_total_k too small
    assert status() == -6
    for cu in ([0, 20, 90], [-4, 20, 23], [0, 23, 20]):                   # bad offsets
        c = kv8_case([100, 30], [20, 3], 4, 2, 64, 16, seed=134)
        c.cu_seqlens_q = torch.tensor(cu, dtype=torch.int32)
        append(attn, c, gpu_cache(c))
        assert status() == -6
        chunk(attn, c, gpu_cache(c))
        assert status() == -6
        attn.attn_kvcache_read_fp8(*gpu_cache(c), dev(c.block_table), dev(c.cu_seqlens_q), 23)
        assert status() == -6


def test_repeatable_captured_and_on_another_stream(attn):
    c = kv8_case([900, 40, 3000], [4, 1, 2], 8, 2, 128, 64, seed=140, rotary_dim=128, spread=0.5)
    cache = gpu_cache(c)
    ins = [dev(t) for t in (c.q, c.k_new, c.v_new)]
    rest = [dev(t) for t in (c.cache_seqlens, c.block_table, c.cu_seqlens_q)]
    tables = [dev(c.rotary_cos), dev(c.rotary_sin)]
    lens = dev(torch.tensor([904, 41, 3002], dtype=torch.int32))

    def step():
        o, l = attn.attn_fwd_kvcache_fp8(*ins, *cache, *rest, 4, 3947, c.scale, True, -1, -1, *tables)
        o2, l2 = attn.attn_decode_kvcache_fp8(o[:3].contiguous(), *cache, lens, rest[1])
        return o, l, o2, l2

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    explicit = attn.attn_decode_kvcache_fp8(want[0][:3].contiguous(), *cache, lens, rest[1], stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want[2:], explicit))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for t in held:
        t.fill_(0)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, held))
    assert attn.attn_get_device_status() == 0


def test_binding_refuses_mismatched_arguments(attn):
    c = kv8_case([30, 40], None, 4, 2, 64, 16, seed=150)
    q, cache = c.q.cuda(), gpu_cache(c)
    sl, bt = dev(c.cache_seqlens), dev(c.block_table)
    f = attn.attn_decode_kvcache_fp8
    for bad in ((q, cache[0], cache[1][:1], *cache[2:], sl, bt),
                (q, *cache[:2], cache[2].transpose(1, 2).contiguous(), cache[3], sl, bt),
                (q[:, :, :32].contiguous(), *cache, sl, bt),
                (q, *cache, sl[:1], bt), (q, *cache, sl, bt[:1]),
                (q.transpose(0, 1), *cache, sl, bt)):
        with pytest.raises(ValueError):
            f(*bad)
    with pytest.raises(TypeError):
        f(q.float(), *cache, sl, bt)
    with pytest.raises(TypeError):
        f(q, *cache, sl.long(), bt)
    with pytest.raises(ValueError):
        f(q, *cache, sl, bt, out=torch.empty(2, 4, 32, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(attn.AttnError):
        f(q, *cache, sl, bt, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        attn.attn_kvcache_read_fp8(*cache, bt, torch.tensor([0, 3, 5], dtype=torch.int32).cuda(), 5,
                                   k=torch.empty(4, 2, 64, dtype=torch.bfloat16, device="cuda"))
