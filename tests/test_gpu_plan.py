"""attn_kvcache_plan against its definition token by token: every output equal."""
import random

import pytest
import torch

from tests import step_exact

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


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(ctx, new, ps, seed, spare=3, width=0):
    """(block table, free list, free count, pages) as lists: held pages in random order, the rest free."""
    old = [-(-c // ps) for c in ctx]
    need = sum(-(-(c + n) // ps) for c, n in zip(ctx, new)) - sum(old)
    pages = sum(old) + need + spare
    perm = list(range(pages))
    random.Random(seed).shuffle(perm)
    width = max([1, width] + [-(-(c + n) // ps) for c, n in zip(ctx, new)])
    table, at = [], 0
    for n in old:
        table.append(perm[at:at + n] + [-7] * (width - n))
        at += n
    return table, perm[at:] + [-5] * (pages - len(perm[at:])), need + spare, pages


def run(attn, ctx, new, ps, seed, pad=0, **kw):
    table, free, count, pages = make(ctx, new, ps, seed, **kw)
    total = sum(new) + pad
    t = ints(table).view(len(ctx), -1)
    got = attn.attn_kvcache_plan(ints(ctx), ints(new), t, ints(free), ints([count]), ps, pages, total)
    want = step_exact.plan(ctx, new, table, free, count, ps, total)
    cu, after, positions, slots, left = (x.tolist() for x in got)
    assert t.tolist() == want[0]
    assert (cu, after, positions, slots, left) == (want[1], want[2], want[3], want[4], [want[5]])
    assert attn.attn_get_device_status() == 0


@pytest.mark.parametrize("ps", [1, 16, 48, 64, 256])
@pytest.mark.parametrize("ctx,new", [
    ([0], [1]),
    ([5], [0]),
    ([0, 0, 0], [0, 0, 0]),
    ([15, 16, 17, 63, 64, 65, 255, 256, 257], [1] * 9),
    ([1, 0, 300, 64], [700, 0, 1, 64]),
    ([1000], [3333]),
])
def test_small_plans(attn, ctx, new, ps):
    for pad in (0, 5, 300):
        run(attn, ctx, new, ps, seed=ps + pad, pad=pad)


@pytest.mark.parametrize("seed", range(8))
def test_random_plans(attn, seed):
    r = random.Random(seed)
    B = r.choice([2, 31, 33, 200, 1023, 1024, 1025, 2500])
    hi = r.choice([1, 3, 40])
    ctx = [r.randint(0, r.choice([1, 50, 500])) for _ in range(B)]
    new = [r.randint(0, hi) for _ in range(B)]
    run(attn, ctx, new, r.choice([1, 16, 64]), seed, pad=r.choice([0, 77]), width=r.choice([0, 40]))


def test_many_tokens_and_many_sequences(attn):
    run(attn, [7, 0, 33], [70000, 1, 60001], 16, seed=1)
    run(attn, [i % 40 for i in range(65535)], [i % 3 for i in range(65535)], 16, seed=2)


@pytest.mark.parametrize("B", [2048, 2049, 65535])
def test_no_tokens_of_many_sequences(attn, B):
    """On both sides of the sizes that take one launch: a step in which nobody has a new token, and a call
    behind it, which would report a launch error that the first left behind."""
    ctx = [i % 40 for i in range(B)]
    run(attn, ctx, [0] * B, 16, seed=5)
    run(attn, [15], [3], 16, seed=6)
    ctx, new, t, free, count = ints(ctx), ints([0] * B), ints([[0, 1, 2]] * B), ints([]), ints([0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        cu, after, positions, slots, left = attn.attn_kvcache_plan(ctx, new, t, free, count, 16, 3, 0)
    graph.replay()
    torch.cuda.synchronize()
    assert not cu.any() and torch.equal(after, ctx) and left.tolist() == [0]
    assert positions.shape == slots.shape == (0,) and (t == ints([0, 1, 2])).all()
    # lengths that do not fit are reported here too
    after = attn.attn_kvcache_plan(ctx, new - 1, t, free, count, 16, 3, 0)[1]
    assert torch.equal(after, ctx) and attn.attn_get_device_status() == -6


def test_no_sequences(attn):
    t = torch.empty((0, 4), dtype=torch.int32, device="cuda")
    e = ints([])
    cu, after, positions, slots, left = attn.attn_kvcache_plan(e, e, t, ints([1, 2]), ints([2]), 16, 9, 3)
    assert cu.tolist() == [0] and positions.tolist() == [0] * 3 and slots.tolist() == [-1] * 3
    assert left.tolist() == [2] and after.numel() == 0


def refused(attn, ctx, new, table, free, count, ps, pages, total):
    t = ints(table)
    cu, after, positions, slots, left = attn.attn_kvcache_plan(
        ints(ctx), ints(new), t, ints(free), ints([count]), ps, pages, total)
    assert attn.attn_get_device_status() == -6
    assert t.tolist() == table and cu.tolist() == [0] * (len(ctx) + 1) and after.tolist() == ctx
    assert positions.tolist() == [0] * total and slots.tolist() == [-1] * total and left.tolist() == [count]


def test_steps_that_do_not_fit_change_nothing(attn):
    good = dict(ctx=[3, 0], new=[2, 20], table=[[7, -1], [-1, -1]], free=[1, 2, 3, 4], count=4, ps=16, pages=9,
                total=22)
    for bad in (dict(count=1), dict(count=-1), dict(count=5), dict(total=21), dict(new=[2, -1]),
                dict(ctx=[-1, 0]), dict(new=[2, 33], total=60), dict(ctx=[2 ** 31 - 1, 0]),
                dict(new=[2, 2 ** 31 - 1])):
        refused(attn, **{**good, **bad})


def test_bad_page_ids_give_their_tokens_no_slot(attn):
    t = ints([[7, -1], [9, -1]])  # page 9 of 9: outside; the last free id as well
    cu, after, positions, slots, left = attn.attn_kvcache_plan(
        ints([15, 3]), ints([3, 1]), t, ints([2, -3]), ints([2]), 16, 9, 4)
    assert attn.attn_get_device_status() == -6
    assert slots.tolist() == [7 * 16 + 15, -1, -1, -1] and positions.tolist() == [15, 16, 17, 3]
    assert t.tolist() == [[7, -1], [9, -1]] and left.tolist() == [1] and cu.tolist() == [0, 3, 4]


def test_in_place_counts_and_lengths_in_a_replayed_graph(attn):
    """Lengths and the free count go on by themselves from replay to replay."""
    B, ps = 5, 16
    ctx, new = [0, 15, 16, 30, 7], [1, 1, 1, 0, 1]
    table, free, count, pages = make(ctx, [40 * n for n in new], ps, seed=4)
    lens, left, t = ints(ctx), ints([count]), ints(table)
    n, f = ints(new), ints(free)
    outs = dict(seqlens_after=lens, free_left=left)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        attn.attn_kvcache_plan(lens.clone(), n, t.clone(), f, left.clone(), ps, pages, 4)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            cu, after, positions, slots, left2 = attn.attn_kvcache_plan(lens, n, t, f, left, ps, pages, 4,
                                                                        **outs)
    torch.cuda.synchronize()
    for _ in range(37):
        graph.replay()
        torch.cuda.synchronize()
        table, cu_w, ctx, pos_w, slots_w, count = step_exact.plan(ctx, new, table, free, count, ps, 4)
        assert (t.tolist(), cu.tolist(), lens.tolist()) == (table, cu_w, ctx)
        assert (positions.tolist(), slots.tolist(), left.tolist()) == (pos_w, slots_w, [count])
    assert B == len(ctx) and after is lens and left2 is left and attn.attn_get_device_status() == 0


def test_given_outputs_streams_and_refusals(attn):
    ctx, new = ints([3, 0]), ints([2, 1])
    t, free, count = ints([[1, -1], [-1, -1]]), ints([4, 5]), ints([2])
    call = lambda **kw: attn.attn_kvcache_plan(*{  # noqa: E731
        **dict(a=ctx, b=new, c=t, d=free, e=count, f=16, g=9, h=3), **kw}.values())
    for bad in (dict(a=ctx.long()), dict(b=ints([1])), dict(c=ints([1, 2])), dict(e=ints([1, 2])),
                dict(d=free.cpu()), dict(a=ints([3, 9, 0, 9])[::2]), dict(h=2 ** 31)):
        with pytest.raises((TypeError, ValueError)):
            call(**bad)
    for bad in (dict(f=0), dict(g=0), dict(h=-1)):
        with pytest.raises(attn.AttnError):
            call(**bad)
    with pytest.raises(ValueError):
        attn.attn_kvcache_plan(ctx, new, t, free, count, 16, 9, 3, positions=ints([0, 0]))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
        late = ints([3, 0]).add_(0)
    got = attn.attn_kvcache_plan(late, new, t, free, count, 16, 9, 3, stream=s)
    s.synchronize()
    assert got[3].tolist() == [19, 20, 80] and attn.attn_get_device_status() == 0
