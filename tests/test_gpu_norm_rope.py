"""Norms of queries and keys with the rotation, their backward pass and the form that writes the paged
cache, against the 64-bit definition."""
import itertools

import pytest
import torch

from exact_attention_70_gb300 import synth
from tests import step_exact
from tests.test_gpu_plan import attn  # noqa: F401

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def rows(gen, T, H, d, scale=1.0):
    return (torch.randn((T, H, d), generator=gen) * scale).to(BF16)


def case(T, Hq, Hkv, d, rot, seed, axes=1, sections=None, mixed=False, inter=False, norm=(True, True),
         w32=False, size=1.0, eps=1e-6, table_rows=97):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn((T, Hq + 2 * Hkv, d), generator=gen) * size).to(BF16)
    c = dict(T=T, Hq=Hq, Hkv=Hkv, d=d, packed=x)
    c["q"], c["k"], c["v"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    c["w"] = [(1 + 0.3 * torch.randn(d, generator=gen)).to(torch.float32 if w32 else BF16) if on else None
              for on in norm]
    cos = sin = pos = None
    if rot:
        cos, sin = synth.rotary_tables(table_rows, rot)
        pos = torch.randint(0, table_rows, (axes, T), generator=gen).int()
    c["how"] = dict(eps=eps, rotary_cos=cos, rotary_sin=sin, positions=pos, rotary_interleaved=inter,
                    sections=sections, sections_interleaved=mixed)
    c["turn"] = step_exact.turn_of(cos, sin, pos, axes, sections, mixed, inter)
    c["gq"], c["gk"] = rows(gen, T, Hq, d), rows(gen, T, Hkv, d)
    return c


def gpu(x):
    return x.cuda() if isinstance(x, torch.Tensor) else x


def parts(c, packed):
    """q, k, v on the GPU, as parts of one tensor or dense."""
    Hq, Hkv = c["Hq"], c["Hkv"]
    if packed:
        x = c["packed"].cuda()
        return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    return tuple(c[n].contiguous().cuda() for n in "qkv")


def how(c):
    return dict(q_weight=gpu(c["w"][0]), k_weight=gpu(c["w"][1]), **{k: gpu(v) for k, v in c["how"].items()})


def check_forward(attn, c, packed=True):  # noqa: F811
    q, k, _ = parts(c, packed)
    qo, ko = attn.attn_qk_norm_rope(q, k, **how(c))
    for got, x, w in ((qo, c["q"], c["w"][0]), (ko, c["k"], c["w"][1])):
        step_exact.within(got, *step_exact.norm_rope(x, w, c["how"]["eps"], c["turn"]))
    assert attn.attn_get_device_status() == 0
    return qo, ko


def check_backward(attn, c, packed=True):  # noqa: F811
    q, k, _ = parts(c, packed)
    got = attn.attn_qk_norm_rope_bwd(gpu(c["gq"]), gpu(c["gk"]), q, k, **how(c))
    for i, (g, x) in enumerate(((c["gq"], c["q"]), (c["gk"], c["k"]))):
        (dx, b), (dw, bw) = step_exact.norm_rope_grad(g, x, c["w"][i], c["how"]["eps"], c["turn"])
        step_exact.within(got[i], dx, b, "dx")
        if dw is None:
            assert got[i + 2] is None
        else:
            step_exact.within(got[i + 2], dw, bw, "dw")
    assert attn.attn_get_device_status() == 0
    return got


CASES = [
    dict(T=1, Hq=1, Hkv=1, d=64, rot=64),
    dict(T=1, Hq=8, Hkv=2, d=128, rot=128, inter=True),
    dict(T=5, Hq=6, Hkv=3, d=64, rot=16, w32=True),
    dict(T=7, Hq=14, Hkv=2, d=128, rot=96),
    dict(T=33, Hq=4, Hkv=4, d=128, rot=64, inter=True, w32=True),
    dict(T=65, Hq=32, Hkv=8, d=128, rot=128),
    dict(T=129, Hq=5, Hkv=1, d=64, rot=48, axes=3, sections=(8, 8, 8)),
    dict(T=100, Hq=12, Hkv=4, d=128, rot=128, axes=3, sections=(16, 24, 24)),
    dict(T=100, Hq=12, Hkv=4, d=128, rot=128, axes=3, sections=(24, 20, 20), mixed=True, inter=True),
    dict(T=64, Hq=3, Hkv=3, d=64, rot=32, axes=2, sections=(9, 7), mixed=True),
    dict(T=64, Hq=2, Hkv=1, d=64, rot=64, axes=2, sections=(5, 27)),
    dict(T=64, Hq=2, Hkv=1, d=128, rot=128, axes=3, sections=(0, 64, 0)),
    dict(T=50, Hq=8, Hkv=8, d=128, rot=0),
    dict(T=50, Hq=8, Hkv=8, d=64, rot=64, norm=(False, False)),
    dict(T=50, Hq=8, Hkv=2, d=128, rot=32, norm=(False, True)),
    dict(T=50, Hq=8, Hkv=2, d=128, rot=32, norm=(True, False), inter=True),
    dict(T=300, Hq=128, Hkv=1, d=64, rot=64),
    dict(T=4099, Hq=7, Hkv=7, d=64, rot=64),
    dict(T=5003, Hq=16, Hkv=4, d=128, rot=128),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_forward(attn, i):  # noqa: F811
    for packed in (True, False):
        check_forward(attn, case(seed=i, **CASES[i]), packed)


@pytest.mark.parametrize("i", range(len(CASES)))
def test_backward(attn, i):  # noqa: F811
    for packed in (True, False):
        check_backward(attn, case(seed=i, **CASES[i]), packed)


@pytest.mark.parametrize("size,eps", [(2.0 ** 100, 1e-6), (2.0 ** 60, 1e-5), (2.0 ** 62, 2.0 ** -64),
                                      (2.0 ** -60, 1e-6), (2.0 ** -20, 1e-12), (2.0 ** -40, 2.0 ** -64),
                                      (0.0, 1e-6)])
def test_rows_of_all_sizes(attn, size, eps):  # noqa: F811
    """Sums of squares past fp32's range, near the border of the second way, lost beside eps, and zero."""
    c = case(40, 6, 2, 128, 64, seed=9, size=size, eps=eps)
    check_forward(attn, c)
    check_backward(attn, c)
    c = case(40, 6, 2, 64, 64, seed=10, size=size, eps=eps)
    c["packed"][::2] = (c["packed"][::2].float() * 2.0 ** -9).to(BF16)  # rows of both ways in a warp
    check_forward(attn, c)
    check_backward(attn, c)


def test_largest_numbers(attn):  # noqa: F811
    c = case(16, 4, 2, 128, 128, seed=11)
    top = torch.finfo(BF16).max
    c["packed"].copy_(torch.where(c["packed"] > 0, top, -top))
    check_forward(attn, c)
    check_backward(attn, c)


@pytest.mark.parametrize("w32", [False, True])
def test_small_rows_under_large_weights(attn, w32):  # noqa: F811
    """rstd w is past fp32's range where x rstd w is not: rows far below one, and of zeros."""
    c = case(40, 6, 2, 128, 64, seed=81, size=2.0 ** -9, eps=1e-12, w32=w32)
    c["packed"][::3] = 0
    c["w"] = [(w.float() * 2.0 ** 120).to(w.dtype) for w in c["w"]]
    check_forward(attn, c)
    top = torch.finfo(BF16).max
    c = case(40, 6, 2, 64, 64, seed=82, size=0.0, w32=w32)
    c["w"] = [torch.where(w > 1, top, -top).to(w.dtype) for w in c["w"]]
    qo, ko = check_forward(attn, c)
    assert not qo.any() and not ko.any()


def test_infinities_and_nan_stay_in_their_rows(attn):  # noqa: F811
    c = case(20, 4, 2, 128, 64, seed=12)
    c["packed"][3, 1, 7] = float("nan")
    c["packed"][8, 4, 100] = float("inf")
    q, k, v = parts(c, True)
    qo, ko = attn.attn_qk_norm_rope(q, k, **how(c))
    assert qo[3, 1].isnan().all() and ko[8, 0, 100].isnan()
    for got, x, w in ((qo, c["q"], c["w"][0]), (ko, c["k"], c["w"][1])):
        y, bound = step_exact.norm_rope(x, w, 1e-6, c["turn"])
        fine = x.float().isfinite().all(-1)
        step_exact.within(got.cpu()[fine], y[fine], bound[fine])
    # without a norm they stay in their planes; elements that do not turn are copied
    qo, ko = attn.attn_qk_norm_rope(q, k, rotary_cos=gpu(c["how"]["rotary_cos"]),
                                    rotary_sin=gpu(c["how"]["rotary_sin"]),
                                    positions=gpu(c["how"]["positions"]))
    assert qo[3, 1].isnan().nonzero().flatten().tolist() == [7, 39]
    assert torch.equal(ko[:, :, 64:], k[:, :, 64:])


@pytest.mark.parametrize("inter,mixed", list(itertools.product([False, True], [False, True])))
def test_one_axis_with_equal_positions_is_three_axes(attn, inter, mixed):  # noqa: F811
    a = case(60, 4, 2, 128, 96, seed=13, inter=inter)
    b = dict(a, how=dict(a["how"], positions=a["how"]["positions"].repeat(3, 1), sections=(16, 16, 16),
                         sections_interleaved=mixed))
    q, k, _ = parts(a, True)
    assert all(torch.equal(x, y) for x, y in zip(attn.attn_qk_norm_rope(q, k, **how(a)),
                                                 attn.attn_qk_norm_rope(q, k, **how(b))))
    g = gpu(a["gq"]), gpu(a["gk"])
    assert all(torch.equal(x, y) for x, y in zip(attn.attn_qk_norm_rope_bwd(*g, q, k, **how(a)),
                                                 attn.attn_qk_norm_rope_bwd(*g, q, k, **how(b))))


def test_in_place(attn):  # noqa: F811
    c = case(77, 6, 2, 64, 32, seed=14)
    q, k, _ = parts(c, False)
    want = attn.attn_qk_norm_rope(q, k, **how(c))
    q2, k2 = q.clone(), k.clone()
    got = attn.attn_qk_norm_rope(q2, k2, q_out=q2, k_out=k2, **how(c))
    assert got[0] is q2 and all(torch.equal(a, b) for a, b in zip(got, want))
    g = gpu(c["gq"]), gpu(c["gk"])
    want = attn.attn_qk_norm_rope_bwd(*g, q, k, **how(c))
    g2 = g[0].clone(), g[1].clone()
    got = attn.attn_qk_norm_rope_bwd(*g2, q, k, dq=g2[0], dk=g2[1], **how(c))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    q2, k2 = q.clone(), k.clone()
    got = attn.attn_qk_norm_rope_bwd(*g, q2, k2, dq=q2, dk=k2, **how(c))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_gradients_as_parts_of_a_projections(attn):  # noqa: F811
    c = case(90, 6, 2, 128, 64, seed=15)
    q, k, _ = parts(c, True)
    g = gpu(c["gq"]), gpu(c["gk"])
    want = attn.attn_qk_norm_rope_bwd(*g, q, k, **how(c))
    whole = torch.full((90, 10, 128), 3.0, dtype=BF16, device="cuda")
    got = attn.attn_qk_norm_rope_bwd(*g, q, k, dq=whole[:, :6], dk=whole[:, 6:8], **how(c))
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and (whole[:, 8:] == 3).all()


def test_repeated_calls_give_the_same_bits(attn):  # noqa: F811
    c = case(3000, 16, 4, 128, 128, seed=16)
    q, k, _ = parts(c, True)
    g = gpu(c["gq"]), gpu(c["gk"])
    first = attn.attn_qk_norm_rope_bwd(*g, q, k, **how(c))
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, attn.attn_qk_norm_rope_bwd(*g, q, k, **how(c))))


def test_gradients_by_differences(attn):  # noqa: F811
    """The gradients against the slope of the 64-bit forward pass along random directions: off by what the
    rounding of dx to bf16 allows, 2^-8 of the sum of |dx v| (and 2^-18 for dw)."""
    c = case(12, 4, 2, 64, 32, seed=17, axes=2, sections=(10, 6), w32=True)
    got = check_backward(attn, c)
    gen = torch.Generator().manual_seed(18)
    for i, name in enumerate("qk"):
        x, w, g = c[name].double(), c["w"][i].double(), c["g" + name].double()
        f = lambda x, w: (step_exact.norm_rope(x, w, 1e-6, c["turn"])[0] * g).sum()  # noqa: E731
        vx, vw = (torch.randn(t.shape, generator=gen, dtype=torch.float64) for t in (x, w))
        h = 1e-6
        slope = (f(x + h * vx, w) - f(x - h * vx, w)) / (2 * h)
        dx = got[i].cpu().double()
        assert abs(slope - (dx * vx).sum()) <= 2.0 ** -7 * (dx * vx).abs().sum()
        slope = (f(x, w + h * vw) - f(x, w - h * vw)) / (2 * h)
        dw = got[i + 2].cpu().double()
        assert abs(slope - (dw * vw).sum()) <= 2.0 ** -10 * (dw * vw).abs().sum()


def test_no_tokens(attn):  # noqa: F811
    c = case(0, 4, 2, 64, 32, seed=19)
    q, k, v = parts(c, False)
    qo, ko = attn.attn_qk_norm_rope(q, k, **how(c))
    assert qo.shape == (0, 4, 64) and ko.shape == (0, 2, 64)
    got = attn.attn_qk_norm_rope_bwd(gpu(c["gq"]), gpu(c["gk"]), q, k, **how(c))
    assert got[0].shape == (0, 4, 64) and not got[2].any() and not got[3].any()
    cache = torch.ones((2, 16, 2, 64), dtype=BF16, device="cuda")
    attn.attn_kvcache_append_norm_rope(q, k, v, cache, cache.clone(), torch.empty(0, dtype=torch.int32, device="cuda"),
                                       **how(c))
    assert (cache == 1).all() and attn.attn_get_device_status() == 0


def append(attn, c, slots, kc, vc, packed=True, **kw):  # noqa: F811
    return attn.attn_kvcache_append_norm_rope(*parts(c, packed), kc, vc, slots, **how(c), **kw)


@pytest.mark.parametrize("i", range(len(CASES)))
def test_append(attn, i):  # noqa: F811
    """Queries and keys have the other call's bits, values their own, slots of no token keep theirs."""
    c = case(seed=40 + i, **CASES[i])
    T, Hkv, d = c["T"], c["Hkv"], c["d"]
    for ps, packed in ((16, True), (3, False), (256, True)):
        pages = -(-T // ps) + 2
        gen = torch.Generator().manual_seed(i)
        slots = torch.randperm(pages * ps, generator=gen)[:T].int()
        if T > 4:
            slots[T // 2] = -1
            slots[T // 3] = -2 ** 31
        kc, vc = rows(gen, pages * ps, Hkv, d).cuda(), rows(gen, pages * ps, Hkv, d).cuda()
        q, k, v = parts(c, packed)
        qw, kw = attn.attn_qk_norm_rope(q, k, **how(c))
        want_k, want_v = kc.clone(), vc.clone()
        on = slots >= 0
        want_k[slots[on].long().cuda()], want_v[slots[on].long().cuda()] = kw[on.cuda()], v[on.cuda()]
        shape = (pages, ps, Hkv, d)
        qo = append(attn, c, slots.cuda(), kc.view(shape), vc.view(shape), packed)
        assert torch.equal(qo, qw) and torch.equal(kc, want_k) and torch.equal(vc, want_v)
    assert attn.attn_get_device_status() == 0


def test_tokens_outside_the_tables_and_the_cache(attn):  # noqa: F811
    c = case(30, 4, 2, 128, 64, seed=70, axes=2, sections=(16, 16))
    want = check_forward(attn, c)
    c["how"]["positions"][0, 4], c["how"]["positions"][1, 9] = -1, 97
    q, k, v = parts(c, True)
    qo, ko = (torch.full(t.shape, 5.0, dtype=BF16, device="cuda") for t in want)
    attn.attn_qk_norm_rope(q, k, q_out=qo, k_out=ko, **how(c))
    assert attn.attn_get_device_status() == -6
    for got, w in ((qo, want[0]), (ko, want[1])):
        assert (got[[4, 9]] == 5).all()
        keep = [t for t in range(30) if t not in (4, 9)]
        assert torch.equal(got[keep], w[keep])
    dq, dk = qo.clone().fill_(5), ko.clone().fill_(5)
    g = gpu(c["gq"]), gpu(c["gk"])
    got = attn.attn_qk_norm_rope_bwd(*g, q, k, dq=dq, dk=dk, **how(c))
    assert attn.attn_get_device_status() == -6
    assert (dq[[4, 9]] == 5).all() and (dk[[4, 9]] == 5).all()
    keep = [t for t in range(30) if t not in (4, 9)]
    h = dict(how(c), positions=how(c)["positions"][:, keep].contiguous())
    less = attn.attn_qk_norm_rope_bwd(g[0][keep], g[1][keep], q[keep].contiguous(), k[keep].contiguous(), **h)
    assert torch.equal(dq[keep], less[0]) and torch.allclose(got[2], less[2], rtol=1e-4, atol=1e-3)
    # slots past the cache
    c = case(30, 4, 2, 128, 64, seed=71)
    kc = torch.zeros((3, 16, 2, 128), dtype=BF16, device="cuda")
    vc = kc.clone()
    slots = torch.arange(30, dtype=torch.int32, device="cuda")
    slots[11], slots[12] = 48, 2 ** 31 - 1
    qo = append(attn, c, slots, kc, vc)
    assert attn.attn_get_device_status() == -6
    qw, kw = attn.attn_qk_norm_rope(*parts(c, True)[:2], **how(c))
    assert torch.equal(qo, qw) and not kc.view(48, 2, 128)[11:13].any() and not vc.view(48, 2, 128)[11:13].any()
    assert torch.equal(kc.view(48, 2, 128)[13:30], kw[13:])


def test_offsets_past_32_bits(attn):  # noqa: F811
    """Tokens of a wide projection and slots of a cache that lie past 2^32 bytes."""
    c = case(40, 4, 2, 128, 64, seed=72)
    want = attn.attn_qk_norm_rope(*parts(c, False)[:2], **how(c))
    stride = 2 ** 26 + 8                          # 40 tokens, 5.4 GB
    big = torch.empty(40 * stride, dtype=BF16, device="cuda").as_strided((40, 8, 128), (stride, 128, 1))
    big.copy_(c["packed"].cuda())
    got = attn.attn_qk_norm_rope(big[:, :4], big[:, 4:6], **how(c))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = attn.attn_qk_norm_rope_bwd(gpu(c["gq"]), gpu(c["gk"]), big[:, :4], big[:, 4:6], dq=big[:, :4],
                                     dk=big[:, 4:6], **how(c))
    want_g = attn.attn_qk_norm_rope_bwd(gpu(c["gq"]), gpu(c["gk"]), *parts(c, False)[:2], **how(c))
    assert all(torch.equal(a, b) for a, b in zip(got, want_g))
    del big, got
    pages = 2 ** 32 // (256 * 2 * 128 * 2) + 3
    kc = torch.empty((pages, 256, 2, 128), dtype=BF16, device="cuda")
    vc = torch.empty((pages, 256, 2, 128), dtype=BF16, device="cuda")
    slots = (pages * 256 - 1 - torch.arange(40, device="cuda")).int()
    append(attn, c, slots, kc, vc)
    assert torch.equal(kc.view(-1, 2, 128)[slots.long()], want[1])
    assert torch.equal(vc.view(-1, 2, 128)[slots.long()], parts(c, False)[2])
    assert attn.attn_get_device_status() == 0


def test_replayed_graphs_and_streams(attn):  # noqa: F811
    c = case(200, 8, 2, 128, 128, seed=73)
    q, k, _ = parts(c, False)
    h = how(c)
    gq, gk = gpu(c["gq"]), gpu(c["gk"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        attn.attn_qk_norm_rope_bwd(gq, gk, q, k, **h)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = attn.attn_qk_norm_rope(q, k, **h) + attn.attn_qk_norm_rope_bwd(gq, gk, q, k, **h)
    torch.cuda.synchronize()
    for seed in (74, 75):
        d = case(200, 8, 2, 128, 128, seed=seed)
        for to, frm in ((q, d["q"]), (k, d["k"]), (gq, d["gq"]), (gk, d["gk"]),
                        (h["positions"], d["how"]["positions"]), (h["q_weight"], d["w"][0])):
            to.copy_(frm)
        graph.replay()
        torch.cuda.synchronize()
        want = attn.attn_qk_norm_rope(q, k, **h) + attn.attn_qk_norm_rope_bwd(gq, gk, q, k, **h)
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    # a stream given: the call follows what stands on it
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
        late = q * 2
    got = attn.attn_qk_norm_rope(late, k, stream=side, **h)
    side.synchronize()
    want = attn.attn_qk_norm_rope(q * 2, k, **h)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and attn.attn_get_device_status() == 0


def test_binding_refusals(attn):  # noqa: F811
    c = case(8, 4, 2, 64, 32, seed=76)
    q, k, v = parts(c, False)
    h = how(c)
    call = lambda q=q, k=k, **kw: attn.attn_qk_norm_rope(q, k, **{**h, **kw})  # noqa: E731
    for bad in (dict(q=q.float()), dict(k=k[:5]), dict(k=k.cpu()), dict(q=q[0]), dict(q=q.transpose(1, 2)),
                dict(q_weight=h["q_weight"][:32]), dict(q_weight=h["q_weight"].half()),
                dict(k_weight=h["k_weight"].float()), dict(positions=None), dict(positions=h["positions"].long()),
                dict(positions=h["positions"][:, :5].contiguous()), dict(sections=(8, 8)),
                dict(rotary_sin=None), dict(q_out=torch.empty_like(k)), dict(k_out=k.transpose(0, 1))):
        with pytest.raises((TypeError, ValueError)):
            call(**bad)
    for bad in (dict(eps=0.0), dict(q=torch.empty((8, 4, 96), dtype=BF16, device="cuda"),
                                    k=torch.empty((8, 2, 96), dtype=BF16, device="cuda"), q_weight=None,
                                    k_weight=None),
                dict(q=q.as_strided((8, 4, 64), (128, 64, 1))),           # tokens that overlap
                dict(q=torch.empty(8 * 260, dtype=BF16, device="cuda").as_strided((8, 4, 64), (260, 64, 1))),
                dict(sections=(17, 0, -1), positions=h["positions"].repeat(3, 1))):
        with pytest.raises(attn.AttnError):
            call(**bad)
    cache = torch.empty((4, 16, 2, 64), dtype=BF16, device="cuda")
    slots = torch.zeros(8, dtype=torch.int32, device="cuda")
    for bad in ((q, k, v[:5], cache, cache, slots), (q, k, v, cache[..., :32], cache, slots),
                (q, k, v, cache, cache[:2], slots), (q, k, v, cache, cache, slots[:5]),
                (q, k, v, cache, cache, slots.long())):
        with pytest.raises((TypeError, ValueError)):
            attn.attn_kvcache_append_norm_rope(*bad, **h)
    # one position per token, without the axis
    a, b = call(positions=h["positions"][0]), call()
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and attn.attn_get_device_status() == 0
