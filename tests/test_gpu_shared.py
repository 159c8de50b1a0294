"""attn_decode_kvcache_shared against the 64-bit definition: every sequence over all its keys through its own
row of the table.  Every slot that no sequence holds is NaN and every table entry that none needs -1."""
import dataclasses
import random

import pytest
import torch

from tests import step_exact
from tests.step_exact import shared_case
from tests.test_gpu_plan import attn  # noqa: F401

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def dev(c):
    return dataclasses.replace(c, **{f.name: getattr(c, f.name).cuda() for f in dataclasses.fields(c)
                                     if isinstance(getattr(c, f.name), torch.Tensor)})


def call(attn, c, **kw):  # noqa: F811
    return attn.attn_decode_kvcache_shared(c.q, c.k_cache, c.v_cache, c.cache_seqlens, c.block_table,
                                           c.group_starts, c.prefix_lens, c.cu_seqlens_q, c.longest, c.scale, **kw)


def by_row(c, lse):
    return lse if c.cu_seqlens_q is None else lse.t()


def check(attn, c, what="", ref=None):  # noqa: F811
    ref = step_exact.shared_exact(c) if ref is None else ref
    out, lse = call(attn, dev(c))
    assert attn.attn_get_device_status() == 0
    n = sum(c.new)
    step_exact.shared_check(out[:n], by_row(c, lse)[:n], [r[:n] for r in ref], what)
    return out, lse


HEADS = [(8, 2, 64, 64), (14, 2, 128, 16), (4, 4, 128, 128), (32, 8, 128, 256), (3, 1, 64, 32), (128, 1, 64, 128),
         (66, 1, 128, 16)]


@pytest.mark.parametrize("heads", range(len(HEADS)))
@pytest.mark.parametrize("prefix", [0, 1, 127, 128, 129, 500, 1024])
def test_decode_of_one_group(attn, heads, prefix):  # noqa: F811
    Hq, Hkv, d, ps = HEADS[heads]
    c = shared_case([(prefix, [(1, 0), (1, 5), (1, 127), (1, 128), (1, 300)])], Hq, Hkv, d, ps, seed=prefix)
    check(attn, c)


@pytest.mark.parametrize("heads", range(len(HEADS)))
def test_groups_of_all_sizes(attn, heads):  # noqa: F811
    """Groups of one sequence, of none, of many; prefixes of none to many keys."""
    Hq, Hkv, d, ps = HEADS[heads]
    c = shared_case([(300, [(1, 40)]), (0, [(1, 3), (1, 200)]), (777, []), (256, [(1, i) for i in range(0, 90, 6)]),
                     (60, [(1, 2), (1, 3)]), (1500, [(1, 0), (1, 1)])], Hq, Hkv, d, ps, seed=7)
    check(attn, c)


@pytest.mark.parametrize("heads", range(len(HEADS)))
def test_chunks(attn, heads):  # noqa: F811
    """None to some hundred new tokens a sequence, a prefix that ends inside a page, rows behind the last."""
    Hq, Hkv, d, ps = HEADS[heads]
    c = shared_case([(333, [(4, 10), (0, 7), (1, 0), (130, 3)]), (130, [(2, 0), (9, 100)]), (500, [(64, 0)])],
                    Hq, Hkv, d, ps, seed=8, padding=5)
    out, lse = check(attn, c)
    keep = torch.full_like(c.q, 3.0).cuda(), torch.full((Hq, c.q.shape[0]), 3.0, device="cuda")
    call(attn, dev(c), out=keep[0], lse=keep[1])
    n = sum(c.new)
    assert torch.equal(keep[0][:n], out[:n]) and torch.equal(keep[1][:, :n], lse[:, :n])
    assert (keep[0][n:] == 3).all() and (keep[1][:, n:] == 3).all()


@pytest.mark.parametrize("Hq,Hkv,d", [(16, 1, 128), (17, 1, 128), (32, 2, 64), (34, 2, 64), (40, 40, 64), (70, 70, 128)])
def test_rows_at_the_border_of_few_and_many_heads(attn, Hq, Hkv, d):  # noqa: F811
    """Units of 16 and 17 rows (the most that count as few, and one more); more kv heads than a warp's lanes."""
    c = shared_case([(300, [(1, 40), (1, 7)]), (0, [(1, 400)])], Hq, Hkv, d, 32, seed=50 + Hq)
    check(attn, c)
    c = shared_case([(300, [(1, 40), (2, 7)]), (0, [(4, 400), (1, 0)])], Hq, Hkv, d, 32, seed=51 + Hq, padding=1)
    check(attn, c)


def test_a_group_that_fills_many_tiles(attn):  # noqa: F811
    c = shared_case([(400, [(1, i % 5) for i in range(150)])], 8, 2, 64, 16, seed=9)       # 600 rows a head
    check(attn, c)
    c = shared_case([(400, [(3, i % 5) for i in range(40)])], 14, 2, 128, 64, seed=10)     # 840
    check(attn, c)


def test_many_groups_and_sequences(attn):  # noqa: F811
    c = shared_case([(130, [(1, 1), (1, 0)])] * 600, 2, 1, 64, 16, seed=11)
    check(attn, c)


def test_more_groups_and_units_than_the_lists_shared_memory_holds(attn):  # noqa: F811
    c = shared_case([(130, [(1, 1), (1, 0)])] * 1100, 1, 1, 64, 16, seed=46)
    check(attn, c)


def test_sequences_that_do_not_have_the_prefix(attn):  # noqa: F811
    """Short and empty sequences in a group, its first one among them, are computed alone."""
    c = shared_case([(300, [(1, None), (1, 4), (1, 9), (1, None), (1, 0)]), (200, [(1, None), (1, 3)]),
                     (200, [(1, None), (1, None)])], 8, 2, 128, 64, seed=12)
    out, lse = check(attn, c)
    assert not out[0].any() and (lse[0] == -float("inf")).all()
    c = shared_case([(300, [(3, None), (5, 4), (2, 9), (0, None), (1, None), (1, 0)])], 8, 2, 64, 32, seed=13)
    check(attn, c)


def test_queries_inside_the_prefix(attn):  # noqa: F811
    """Sequences whose new tokens begin before the prefix ends see it only in part."""
    c = shared_case([(300, [(4, 20), (4, 0), (4, 1)])], 8, 2, 128, 64, seed=14, decode=False)
    ref = step_exact.shared_exact(c)
    for prefix in (300, 301, 302, 303, 304, 305):  # what the sequences have in common does not end with it
        c.prefix_lens[0] = prefix
        for b in (1, 2):
            if prefix > 300:  # (copies of keys 300 .. prefix - 1 of the first sequence)
                for t in (c.k_cache, c.v_cache):
                    for j in range(300, min(prefix, c.keys[b])):
                        t[c.block_table[b, j // 64], j % 64] = t[c.block_table[0, j // 64], j % 64]
        ref = step_exact.shared_exact(c)
        check(attn, c, prefix, ref)


def test_a_prefix_that_no_sequence_has(attn):  # noqa: F811
    """Prefixes longer than the sequences, and than the table holds: every sequence is computed alone."""
    c = shared_case([(0, [(1, 40), (1, 300), (2, 0)]), (5000, []), (0, [(1, 9)])], 8, 2, 64, 16, seed=47)
    ref = step_exact.shared_exact(c)
    for prefix in (304, 10 ** 6, 2 ** 31 - 1):
        c.prefix_lens[:] = prefix
        check(attn, c, prefix, ref)


def test_no_keys_at_all(attn):  # noqa: F811
    c = shared_case([(0, [(1, None), (1, None)])], 8, 2, 64, 16, seed=15)
    check(attn, c)
    c = shared_case([(0, [(0, 0)])], 8, 2, 64, 16, seed=16, decode=False, padding=2)
    check(attn, c)


def test_a_step_without_tokens(attn):  # noqa: F811
    """max_seqlen_q 0, only padding: nothing to do, and nothing is written."""
    c = shared_case([(200, [(0, 7), (0, 9)])], 8, 2, 64, 16, seed=16, decode=False, padding=3)
    c.longest = 0
    out, lse = torch.full_like(c.q, 3.0).cuda(), torch.full((8, 3), 3.0, device="cuda")
    call(attn, dev(c), out=out, lse=lse)
    assert attn.attn_get_device_status() == 0
    assert (out == 3).all() and (lse == 3).all()


def test_more_queries_than_keys(attn):  # noqa: F811
    """Rows that stand before the first key see nothing."""
    c = shared_case([(0, [(5, 0), (3, 2)])], 8, 2, 64, 16, seed=17, decode=False)
    c.cache_seqlens[0] = 2
    c.keys[0] = 2
    check(attn, c)


def test_without_groups(attn):  # noqa: F811
    c = shared_case([(300, [(1, 40), (1, 700), (1, 0)])], 8, 2, 128, 64, seed=18)
    ref = step_exact.shared_exact(c)
    g = dev(c)
    out, lse = attn.attn_decode_kvcache_shared(g.q, g.k_cache, g.v_cache, g.cache_seqlens, g.block_table,
                                               softmax_scale=c.scale)
    step_exact.shared_check(out, lse, ref)
    o2, l2 = attn.attn_decode_kvcache(g.q, g.k_cache, g.v_cache, g.cache_seqlens, g.block_table, c.scale)
    assert (out.float() - o2.float()).abs().max() < 0.02 and (lse - l2).abs().max() < 1e-4
    assert attn.attn_get_device_status() == 0


@pytest.mark.filterwarnings("ignore:DEBUG")
@pytest.mark.parametrize("Hq,Hkv,new,few", [(8, 2, 1, True), (32, 8, 4, True), (16, 1, 1, True), (6, 2, 5, True),
                                            (17, 1, 1, False), (32, 8, 5, False), (6, 2, 6, False)])
def test_without_groups_and_few_rows_a_sequence(attn, tmp_path, Hq, Hkv, new, few):  # noqa: F811
    """However many sequences there are, no unit has more rows than a sequence: up to 16 take the kernel for few
    rows.  An empty group list and groups without a prefix give the same bits."""
    seqs = [(1 + i % new, None if i == 3 else 37 * i) for i in range(23)]
    c = shared_case([(0, seqs)], Hq, Hkv, 64, 32, seed=70 + new)
    want = check(attn, c)
    c = dev(c)
    none = dataclasses.replace(c, group_starts=None, prefix_lens=None)
    starts, lens = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (1, 0))
    empty = dataclasses.replace(c, group_starts=starts, prefix_lens=lens)
    for x in (call(attn, none), call(attn, empty)):
        assert all(torch.equal(a, b) for a, b in zip(want, x))
    graph = torch.cuda.CUDAGraph(keep_graph=True)  # (its dump names the kernels)
    graph.enable_debug_mode()
    with torch.cuda.graph(graph):
        call(attn, none)
    graph.debug_dump(str(tmp_path / "graph"))
    text = (tmp_path / "graph").read_text()
    assert "shared_units_kernel" in text
    assert ("shared_small_kernel" in text) == few and ("shared_attn_kernel" in text) != few
    assert attn.attn_get_device_status() == 0


@pytest.mark.parametrize("scale,size", [(1e-6, 1.0), (3.0, 1.0), (0.1, 30.0), (2.0 ** -100, 1.0)])
def test_scales(attn, scale, size):  # noqa: F811
    """Flat and sharp weights; rows whose maximum moves from block to block."""
    c = shared_case([(700, [(1, 9), (1, 300), (2, 40)])], 8, 2, 128, 64, seed=19, scale=scale, size=size)
    check(attn, c)


def test_rising_and_falling_scores(attn):  # noqa: F811
    for sign in (1, -1):
        c = shared_case([(1000, [(1, 400), (1, 1)])], 4, 2, 64, 16, seed=20)
        pos = torch.arange(1401)
        for b in (0, 1):
            j = pos[:c.keys[b]]
            row = c.block_table[b].long()[j // 16], j % 16
            c.k_cache[row] = (sign * j[:, None, None] * 0.01 + 0.1 * c.k_cache[row].float()).to(BF16)
        c.q.fill_(1.0)
        check(attn, c)


def test_a_prefix_through_one_row(attn):  # noqa: F811
    """The other sequences' entries for the prefix's pages are not looked at."""
    c = shared_case([(300, [(1, 10), (1, 100), (1, 20)])], 8, 2, 128, 64, seed=21)
    ref = step_exact.shared_exact(c)
    c.block_table[1:, :300 // 64] = -9
    check(attn, c, ref=ref)


def test_nan_behind_and_before_a_sequences_keys(attn):  # noqa: F811
    """In its own copy of the page that the prefix ends in, what stands before the end is not looked at."""
    c = shared_case([(330, [(1, 10), (1, 100), (1, 20)])], 8, 2, 64, 256, seed=22)
    ref = step_exact.shared_exact(c)
    for b in (1, 2):
        c.k_cache[c.block_table[b, 1], :330 - 256] = float("nan")
        c.v_cache[c.block_table[b, 1], :330 - 256] = float("inf")
    check(attn, c, ref=ref)


def test_nan_keys_reach_the_rows_that_see_them(attn):  # noqa: F811
    c = shared_case([(300, [(1, 10), (1, 100)]), (300, [(1, 10), (1, 100)])], 8, 2, 64, 64, seed=23)
    want, want_lse = call(attn, dev(c))
    c.k_cache[c.block_table[0, 2], 5, 1, 3] = float("nan")  # the first group's prefix, kv head 1
    c.k_cache[c.block_table[3, 5], 60, 0, 3] = float("nan")  # the last sequence's key 380, kv head 0
    out, lse = call(attn, dev(c))
    assert out[:2, 4:].isnan().all() and lse[:2, 4:].isnan().all()
    assert out[3, :4].isnan().all() and lse[3, :4].isnan().all()
    for rows, heads in ((slice(0, 2), slice(0, 4)), (2, slice(None)), (3, slice(4, 8))):
        assert torch.equal(out[rows, heads], want[rows, heads]) and torch.equal(lse[rows, heads], want_lse[rows, heads])


@pytest.mark.parametrize("seed", range(24))
def test_random_configurations(attn, seed):  # noqa: F811
    r = random.Random(seed)
    Hkv = r.choice([1, 2, 3, 8])
    Hq, d, ps = Hkv * r.choice([1, 2, 4, 5, 7, 8]), r.choice([64, 128]), r.choice([16, 32, 64, 128, 256])
    top = r.choice([1, 1, 6])
    groups = []
    for _ in range(r.randint(1, 5)):
        p = r.choice([0, r.randint(1, 300), r.randint(100, 3000)])
        seqs = [(r.randint(1, top) if top > 1 else 1, r.choice([None, 0, r.randint(0, 50), r.randint(0, 900)]))
                for _ in range(r.randint(0, 9))]
        groups.append((p, seqs))
    groups.append((r.randint(0, 500), [(1, 5)]))
    check(attn, shared_case(groups, Hq, Hkv, d, ps, seed=seed, decode=top == 1), (seed, groups))


@pytest.mark.parametrize("groups,Hq,Hkv,d", [
    ([(150, [(1, 300 + 3 * i) for i in range(120)])], 8, 8, 64),                     # few rows: most of the work
    ([(4000, [(1, 20 * (i % 7)) for i in range(40)])] * 2, 8, 2, 128),               # few rows: a small part of it
    ([(700, [(1, 90 * (i % 5)) for i in range(20)])] * 24, 8, 8, 64),                # more tiles than CTAs
    ([(260, [(17, 30)] * 3 + [(1, 500)] * 30), (200, [(2, 5)] * 30)], 4, 4, 128)],   # both kinds among the own keys
    ids=["few", "many", "tiles", "own"])
def test_units_of_both_kinds(attn, groups, Hq, Hkv, d):  # noqa: F811
    decode = all(n == 1 for _, seqs in groups for n, _ in seqs)
    c = shared_case(groups, Hq, Hkv, d, 16, seed=60, decode=decode)
    out, lse = check(attn, c)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip((out, lse), call(attn, dev(c))))


def test_a_long_prefix_in_many_pieces(attn):  # noqa: F811
    c = shared_case([(20011, [(1, 3), (1, 2000), (1, 77)])], 4, 2, 128, 64, seed=24)
    check(attn, c)


def test_same_bits_again(attn):  # noqa: F811
    c = dev(shared_case([(3000, [(1, i) for i in range(40)])], 16, 4, 128, 64, seed=25))
    first = call(attn, c)
    for _ in range(10):
        assert all(torch.equal(a, b) for a, b in zip(first, call(attn, c)))


def test_pages_past_32_bit_offsets(attn):  # noqa: F811
    c = dev(shared_case([(200, [(1, 9), (1, 300), (2, 40)])], 8, 8, 128, 16, seed=26))
    want = call(attn, c)
    shift = 2 ** 32 // (16 * 8 * 128 * 2) + 5
    for name in ("k_cache", "v_cache"):
        near = getattr(c, name)
        far = torch.empty((shift + near.shape[0], *near.shape[1:]), dtype=BF16, device="cuda")
        far[shift:].copy_(near)
        setattr(c, name, far)
    c.block_table = torch.where(c.block_table >= 0, c.block_table + shift, c.block_table).int()
    assert all(torch.equal(a, b) for a, b in zip(want, call(attn, c)))
    assert attn.attn_get_device_status() == 0


def test_replayed_graph_with_other_lengths(attn):  # noqa: F811
    """A captured decode step whose lengths, tables and groups change between replays."""
    make = lambda seed: shared_case(  # noqa: E731
        [(p, [(1, random.Random(seed + b).randint(0, 600)) for b in range(n)])
         for p, n in (((600, 3), (300, 5)) if seed % 2 else ((100, 6), (2000, 2)))], 8, 2, 128, 64, seed=seed)
    cases = [make(s) for s in range(30, 34)]
    pages = max(c.k_cache.shape[0] for c in cases)
    width = max(c.block_table.shape[1] for c in cases)
    buf = dev(cases[0])
    buf.k_cache = torch.zeros((pages, 64, 2, 128), dtype=BF16, device="cuda")
    buf.v_cache = torch.zeros_like(buf.k_cache)
    buf.block_table = torch.full((8, width), -1, dtype=torch.int32, device="cuda")

    def load(c):
        for name in ("q", "cache_seqlens", "group_starts", "prefix_lens"):
            getattr(buf, name).copy_(getattr(c, name))
        n, w = c.k_cache.shape[0], c.block_table.shape[1]
        buf.k_cache[:n], buf.v_cache[:n] = c.k_cache.cuda(), c.v_cache.cuda()
        buf.block_table[:, :w] = c.block_table.cuda()

    load(cases[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(attn, buf)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out, lse = call(attn, buf)
    torch.cuda.synchronize()
    for c in cases[1:] + cases[:1]:
        load(c)
        graph.replay()
        torch.cuda.synchronize()
        step_exact.shared_check(out, lse, step_exact.shared_exact(c))
    assert attn.attn_get_device_status() == 0


def test_two_streams_at_once(attn):  # noqa: F811
    a = dev(shared_case([(3000, [(1, 100 * i) for i in range(9)])], 8, 2, 128, 64, seed=40))
    b = dev(shared_case([(700, [(3, 50), (2, 9)])], 14, 2, 64, 16, seed=41))
    want = call(attn, a), call(attn, b)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    got = [(call(attn, a, stream=s), call(attn, b, stream=t)) for _ in range(20)]
    torch.cuda.synchronize()
    for x in got:
        assert all(torch.equal(p, q) for w, g in zip(want, x) for p, q in zip(w, g))


def test_what_stands_before_on_the_stream(attn):  # noqa: F811
    c = dev(shared_case([(500, [(1, 30), (1, 3)])], 8, 2, 64, 16, seed=42))
    want = call(attn, c)
    s = torch.cuda.Stream()
    late = dataclasses.replace(c)
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
        late.q, late.k_cache, late.cache_seqlens = c.q + 0, c.k_cache + 0, c.cache_seqlens + 0
    got = call(attn, late, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_lengths_that_do_not_fit(attn):  # noqa: F811
    """Nothing is written, the status says so, and the next call is right."""
    good = shared_case([(300, [(2, 40), (1, 7)]), (130, [(1, 0)])], 8, 2, 64, 16, seed=43)
    want = call(attn, dev(good))
    width = good.block_table.shape[1] * 16
    for bad in (dict(cache_seqlens=[342, -1, 131]), dict(cache_seqlens=[342, width + 1, 131]),
                dict(group_starts=[0, 2, 4]), dict(group_starts=[0, 2, 2]), dict(group_starts=[1, 2, 3]),
                dict(group_starts=[0, 4, 3]), dict(group_starts=[0, -1, 3]), dict(prefix_lens=[-1, 130]),
                dict(cu_seqlens_q=[0, 3, 2, 4]), dict(cu_seqlens_q=[0, 2, 3, 5]),
                dict(cu_seqlens_q=[-1, 2, 3, 4]), dict(longest=1)):
        c = dataclasses.replace(good, **{k: torch.tensor(v, dtype=torch.int32) if isinstance(v, list) else v
                                         for k, v in bad.items()})
        out, lse = torch.full_like(c.q, 3.0).cuda(), torch.full((8, 4), 3.0, device="cuda")
        call(attn, dev(c), out=out, lse=lse)
        assert attn.attn_get_device_status() == -6, bad
        assert (out == 3).all() and (lse == 3).all(), bad
        assert all(torch.equal(a, b) for a, b in zip(want, call(attn, dev(good))))
    assert attn.attn_get_device_status() == 0


def test_bad_pages(attn):  # noqa: F811
    """A page outside the cache raises the status; sequences that do not read it keep their results."""
    c = shared_case([(300, [(1, 40), (1, 7)]), (200, [(1, 9), (1, 30)])], 8, 2, 64, 16, seed=44)
    want = call(attn, dev(c))
    for page in (-1, c.k_cache.shape[0], 2 ** 31 - 1, -2 ** 31):
        d = dataclasses.replace(c, block_table=c.block_table.clone())
        d.block_table[1, 300 // 16] = page
        out, lse = call(attn, dev(d))
        assert attn.attn_get_device_status() == -6
        keep = [0, 2, 3]
        assert torch.equal(out[keep], want[0][keep]) and torch.equal(lse[keep], want[1][keep])


def test_binding_refusals(attn):  # noqa: F811
    c = dev(shared_case([(30, [(1, 4), (1, 7)])], 8, 2, 64, 16, seed=45))
    f = lambda **kw: call(attn, dataclasses.replace(c, **kw))  # noqa: E731
    for bad in (dict(q=c.q.float()), dict(q=c.q[:1]), dict(k_cache=c.k_cache[:, :, :1]), dict(v_cache=c.v_cache[1:]),
                dict(cache_seqlens=c.cache_seqlens[:1]), dict(block_table=c.block_table[0]),
                dict(group_starts=c.group_starts[:1]), dict(prefix_lens=None), dict(prefix_lens=c.prefix_lens.cpu()),
                dict(cu_seqlens_q=c.group_starts), dict(q=c.q[:, ::2])):
        with pytest.raises((TypeError, ValueError)):
            f(**bad)
    with pytest.raises(attn.AttnError):
        f(scale=0.0)
    with pytest.raises(ValueError):
        call(attn, c, out=c.q[:1])
    with pytest.raises(ValueError):
        call(attn, c, lse=torch.empty((8, 2), device="cuda"))
    with pytest.raises(attn.AttnError):
        call(attn, c, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    ws = torch.empty(attn.attn_decode_kvcache_shared_workspace_bytes(2, 1, 2, 8, 2, 64), dtype=torch.uint8,
                     device="cuda")
    assert all(torch.equal(a, b) for a, b in zip(call(attn, c), call(attn, c, workspace=ws)))
    assert attn.attn_get_device_status() == 0
