"""Calls on the 8-bit paged KV cache that its documentation allows beside the plain ones: pages past
32-bit offsets, pages shared by sequences, two streams at once, captured graphs whose lengths and
tokens change between replays, offsets at the ends of their type."""
import pytest
import torch

from tests import kv8_exact
from tests.kv8_exact import kv8_case
from tests.test_gpu_kv8 import append, attn, chunk, dev, gpu_cache, same_cache  # noqa: F401

pytestmark = pytest.mark.gpu


def test_pages_past_32_bit_offsets(attn):  # noqa: F811
    """The same tokens in pages whose bytes start past 2^32 give the same bits."""
    shift = 2 ** 32 // (16 * 8 * 128) + 5                    # pages of 16 tokens, 8 heads, d 128
    c = kv8_case([200, 33, 0], [5, 40, 3], 16, 8, 128, 16, seed=300, rotary_dim=128)
    pages = c.k_cache.shape[0]
    near = gpu_cache(c)
    far = []
    for t in near:
        big = torch.empty(shift + pages, *t.shape[1:], dtype=torch.uint8, device="cuda")
        big[shift:].copy_(t)
        far.append(big)
    assert far[0][shift:].data_ptr() - far[0].data_ptr() >= 2 ** 32
    want = chunk(attn, c, near)
    lens = c.cache_seqlens + torch.tensor(c.new, dtype=torch.int32)
    q = dev(c.q[:3])
    want_d = attn.attn_decode_kvcache_fp8(q, *near, dev(lens), dev(c.block_table))
    cu = dev(torch.tensor([0, 205, 278, 281], dtype=torch.int32))
    want_r = attn.attn_kvcache_read_fp8(*near, dev(c.block_table), cu, 281)
    c.block_table = torch.where(c.block_table >= 0, c.block_table + shift, c.block_table)
    got = chunk(attn, c, far)
    got_d = attn.attn_decode_kvcache_fp8(q, *far, dev(lens), dev(c.block_table))
    got_r = attn.attn_kvcache_read_fp8(*far, dev(c.block_table), cu, 281)
    for a, b in zip((*want, *want_d, *want_r, *near), (*got, *got_d, *got_r, *[t[shift:] for t in far])):
        assert torch.equal(a, b)
    assert attn.attn_get_device_status() == 0


def test_sequences_that_share_a_prefix(attn):  # noqa: F811
    """Three sequences on the same four pages, each going on in a page of its own: the results are
    those of copies."""
    c = kv8_case([256, 256, 256], [3, 1, 9], 8, 2, 64, 64, seed=310, rotary_dim=64)
    table = c.block_table.clone()
    cache = gpu_cache(c)
    for t in cache:                                          # every sequence holds sequence 0's prefix
        for b in (1, 2):
            t[table[b, :4].long().cuda()] = t[table[0, :4].long().cuda()]
    copies = [t.clone() for t in cache]
    want = chunk(attn, c, copies)
    c.block_table[1:, :4] = table[0, :4]
    got = chunk(attn, c, cache)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    lens = dev(torch.tensor([259, 257, 265], dtype=torch.int32))
    want = attn.attn_decode_kvcache_fp8(dev(c.q[:3]), *copies, lens, dev(table))
    got = attn.attn_decode_kvcache_fp8(dev(c.q[:3]), *cache, lens, dev(c.block_table))
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert attn.attn_get_device_status() == 0


@pytest.mark.parametrize("new", [[4, 1], [300, 120]])        # on the codes; staged
def test_two_streams_at_once(attn, new):  # noqa: F811
    cases = [kv8_case([3000, 500], new, 32, 8, 128, 64, seed=320 + i, rotary_dim=128) for i in range(2)]
    caches = [gpu_cache(c) for c in cases]
    want = [chunk(attn, c, k) for c, k in zip(cases, caches)]
    ins = [([dev(t) for t in (c.q, c.k_new, c.v_new)],
            [dev(t) for t in (c.cache_seqlens, c.block_table, c.cu_seqlens_q)],
            [dev(t) for t in (c.rotary_cos, c.rotary_sin)]) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            a, b, r = ins[i]
            got[i].append(attn.attn_fwd_kvcache_fp8(*a, *caches[i], *b, max(new), 3500 + sum(new),
                                                    cases[i].scale, True, -1, -1, *r, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for o, l in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])
    assert attn.attn_get_device_status() == 0


@pytest.mark.parametrize("rotary", [0, 128])
@pytest.mark.parametrize("new", [[4, 1, 0], [260, 7, 130]])  # on the codes; staged
def test_graph_replayed_with_other_tokens(attn, new, rotary):  # noqa: F811
    """One captured chunk and decode, replayed after its inputs, lengths and offsets changed."""
    first = kv8_case([900, 40, 1500], new, 32, 8, 128, 64, seed=330, rotary_dim=rotary)
    later = kv8_case([870, 3, 1450], new[::-1], 32, 8, 128, 64, seed=331, rotary_dim=rotary)
    pages = max(first.k_cache.shape[0], later.k_cache.shape[0])
    width = max(first.block_table.shape[1], later.block_table.shape[1])

    def padded(t, n, value):
        return torch.cat((t, torch.full((n - t.shape[0], *t.shape[1:]), value, dtype=t.dtype)))

    rows = max(x.rotary_cos.shape[0] for x in (first, later)) if rotary else 0

    def inputs(c):
        table = torch.full((3, width), -1, dtype=torch.int32)
        table[:, :c.block_table.shape[1]] = c.block_table
        out = [c.q, c.k_new, c.v_new, *(padded(t, pages, 255) for t in c.cache), c.cache_seqlens, table,
               c.cu_seqlens_q]
        if rotary:
            out += [padded(c.rotary_cos, rows, 1.0), padded(c.rotary_sin, rows, 0.0)]
        return out

    held = [t.cuda() for t in inputs(first)]

    def step():
        q, k, v, kc, vc, ks, vs, sl, bt, cu = held[:10]
        o, l = attn.attn_fwd_kvcache_fp8(q, k, v, kc, vc, ks, vs, sl, bt, cu, max(new), 4000, 128 ** -0.5,
                                         True, -1, -1, *held[10:])
        lens = sl + cu[1:] - cu[:-1]
        return o, l, *attn.attn_decode_kvcache_fp8(q[:3].contiguous(), kc, vc, ks, vs, lens, bt)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for c in (later, first, later):
        for h, t in zip(held, inputs(c)):
            h.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        arrays = kv8_exact.appended(c)
        same_cache([t[:n.shape[0]] for t, n in zip(held[3:7], arrays)], arrays)
        kv8_exact.check(got[0], got[1].t(), kv8_exact.attention(c, arrays), 2.0 ** -11, rotary > 0, "replay")
        for h, t in zip(held, inputs(c)):
            h.copy_(t)
        assert all(torch.equal(a, b) for a, b in zip(got, step()))
    assert attn.attn_get_device_status() == 0


def test_offsets_at_the_ends_of_their_type(attn):  # noqa: F811
    c = kv8_case([100, 30], [20, 3], 4, 2, 64, 16, seed=340)
    low, high = -2 ** 31, 2 ** 31 - 1
    for cu in ([low, 20, 23], [low, low, high], [0, high, low], [low, high, 23], [high, high, high]):
        c.cu_seqlens_q = torch.tensor(cu, dtype=torch.int32)
        append(attn, c, gpu_cache(c))
        assert attn.attn_get_device_status() == -6
        chunk(attn, c, gpu_cache(c))
        assert attn.attn_get_device_status() == -6
        attn.attn_kvcache_read_fp8(*gpu_cache(c), dev(c.block_table), dev(c.cu_seqlens_q), 23)
        assert attn.attn_get_device_status() == -6
    c = kv8_case([100, 30], [200, 3], 32, 16, 64, 16, seed=341, rotary_dim=64)        # staged
    for cu in ([low, 200, 203], [0, high, low], [low, high, 203]):
        c.cu_seqlens_q = torch.tensor(cu, dtype=torch.int32)
        chunk(attn, c, gpu_cache(c))
        assert attn.attn_get_device_status() == -6


def test_binding_refuses_what_a_c_int_or_a_workspace_cannot_hold(attn):  # noqa: F811
    c = kv8_case([30, 40], [3, 4], 4, 2, 64, 16, seed=350)
    cache = gpu_cache(c)
    for bad in (dict(max_total_k=2 ** 32), dict(window=(2 ** 31, -1)), dict(window=(-1, 2 ** 40))):
        with pytest.raises(ValueError):
            chunk(attn, c, cache, **bad)
    one = torch.empty(256, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        chunk(attn, c, cache, workspace=one[:1].expand(1 << 24))
    with pytest.raises(ValueError):
        attn.attn_decode_kvcache_fp8(dev(c.q[:2]), *cache, dev(c.cache_seqlens), dev(c.block_table),
                                     workspace=one[:1].expand(1 << 24))
    same_cache(cache, [t.numpy() for t in c.cache])
