"""CPU checks of the step's calls: their 64-bit definitions by hand, and what the C ABI and the binding
refuse before touching a device."""
import ctypes

import pytest
import torch

from exact_attention_70_gb300 import binding
from exact_attention_70_gb300 import build as attn_build
from tests import step_exact
from tests.test_kv8_host import refusals

P = ctypes.c_void_p
FAKE = P(4096)  # never dereferenced: every call below fails validation first
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    attn_build.build()
    return binding.load()


def ints(*n):
    return (ctypes.c_int32 * len(n))(*n)


def test_plan_by_hand():
    got = step_exact.plan([3, 0, 4], [2, 3, 0], [[7, -1], [-1, -1], [9, -1]], [4, 5, 6], 3, 4, 7)
    table, cu, after, positions, slots, left = got
    assert table == [[7, 6], [5, -1], [9, -1]] and cu == [0, 2, 5, 5] and after == [5, 3, 4]
    assert positions == [3, 4, 0, 1, 2, 0, 0] and slots == [31, 24, 20, 21, 22, -1, -1] and left == 1


def test_plane_axes_by_hand():
    assert step_exact.plane_axes(8, 3, (2, 3, 3), False) == [0, 0, 1, 1, 1, 2, 2, 2]
    assert step_exact.plane_axes(8, 3, (4, 2, 2), True) == [0, 1, 2, 0, 1, 2, 0, 0]
    assert step_exact.plane_axes(8, 2, (5, 3), True) == [0, 1, 0, 1, 0, 1, 0, 0]


def test_gradients_of_the_definition_are_those_of_differences():
    gen = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    for inter in (False, True):
        x, w, g = rnd(3, 2, 64), 1 + 0.1 * rnd(64), rnd(3, 2, 64)
        ang = rnd(3, 1, 16)
        turn = step_exact.Turn(ang.cos(), ang.sin(), inter)
        f = lambda x, w: (step_exact.norm_rope(x, w, 1e-3, turn)[0] * g).sum()  # noqa: E731
        (dx, _), (dw, _) = step_exact.norm_rope_grad(g, x, w, 1e-3, turn)
        for _ in range(3):
            vx, vw, h = rnd(3, 2, 64), rnd(64), 1e-5
            assert abs((f(x + h * vx, w) - f(x - h * vx, w)) / (2 * h) - (dx * vx).sum()) < 1e-6
            assert abs((f(x, w + h * vw) - f(x, w - h * vw)) / (2 * h) - (dw * vw).sum()) < 1e-6


def test_plan_refusals(lib):
    names = ["sl", "new", "bt", "free", "count", "left", "cu", "after", "pos", "slots", "batch", "total", "ps",
             "mp", "nfree", "np", "ws", "wsb", "stream"]
    call = refusals(lib.attn_kvcache_plan, names,
                    [FAKE] * 10 + [2, 4000, 16, 4, 8, 16, FAKE, 1 << 20, None])
    for name in names[:10]:
        assert call(**{name: None}) == -1, name
        assert call(**{name: P(4098)}) == -1, name
    for bad in (dict(batch=-1), dict(total=-1), dict(ps=0), dict(mp=0), dict(nfree=-1), dict(np=0)):
        assert call(**bad) == -1
    assert call(batch=65536) == -2
    assert call(np=1 << 28) == -2                # slots past 31 bits
    assert call(mp=1 << 27) == -2                # positions past 2^30
    assert call(ws=None) == -3
    assert call(wsb=16) == -3
    assert call(ws=P(4096 + 16)) == -3
    assert binding.attn_kvcache_plan_workspace_bytes(64, 4000) == 512
    assert binding.attn_kvcache_plan_workspace_bytes(3000, 0) == 12032
    assert binding.attn_kvcache_plan_workspace_bytes(64, 64) == 0
    assert binding.attn_kvcache_plan_workspace_bytes(70000, 64) == 0


HOW = ["qw", "kw", "w32", "eps", "cos", "sin", "rot", "rows", "inter", "pos", "axes", "sections", "mixed"]
HOW_GOOD = [FAKE, FAKE, 0, 1e-6, FAKE, FAKE, 64, 9, 0, FAKE, 1, None, 0]


def norm_rope_refusals(call):
    for bad in (dict(total=-1), dict(hq=0), dict(hkv=0), dict(q=None), dict(k=None), dict(q=P(4104)),
                dict(k=P(4104)), dict(qs=8 * 128 - 8), dict(ks=2 * 128 + 4), dict(qs=1 << 32),
                dict(eps=0.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(eps=1e-20),
                dict(eps=-1.0), dict(cos=None), dict(sin=None), dict(rows=0), dict(pos=None),
                dict(pos=P(4097)), dict(cos=P(4104)), dict(axes=0), dict(qw=P(4097)),
                dict(kw=P(4098), w32=1), dict(axes=2), dict(axes=2, sections=ints(16, 17)),
                dict(axes=2, sections=ints(33, -1)), dict(axes=3, sections=ints(2 ** 30, 2 ** 30, 2 ** 31 - 1)),
                dict(axes=2, sections=ints(15, 17), mixed=1),  # axis 1 gets every other plane: 16 at most
                dict(axes=3, sections=ints(8, 12, 12), mixed=1)):
        assert call(**bad) == -1, bad
    for bad in (dict(d=96), dict(rot=24), dict(rot=144), dict(rot=-16), dict(axes=4, sections=ints(8, 8, 8, 8)),
                dict(hq=65536), dict(total=1 << 29)):
        assert call(**bad) == -2, bad
    assert call(total=0) == 0
    assert call(total=0, q=None, k=None) == 0
    # sections that come out
    assert call(total=0, axes=2, sections=ints(16, 16), mixed=1) == 0
    assert call(total=0, axes=3, sections=ints(12, 10, 10), mixed=1) == 0
    assert call(total=0, axes=3, sections=ints(0, 32, 0)) == 0


def test_norm_rope_refusals(lib):
    names = ["q", "k", "qs", "ks"] + HOW + ["qo", "ko", "total", "hq", "hkv", "d", "stream"]
    call = refusals(lib.attn_qk_norm_rope, names,
                    [FAKE, FAKE, 1536, 1536] + HOW_GOOD + [None, FAKE, 5, 8, 2, 128, None])
    norm_rope_refusals(call)
    assert call() == -1                          # no q_out
    assert call(qo=P(4104)) == -1


def test_sections_of_one_axis_have_all_planes(lib):
    """One axis needs no sections; those given have to come out all the same."""
    names = ["q", "k", "qs", "ks"] + HOW + ["qo", "ko", "total", "hq", "hkv", "d", "stream"]
    call = refusals(lib.attn_qk_norm_rope, names,
                    [FAKE, FAKE, 1536, 1536] + HOW_GOOD + [FAKE, FAKE, 0, 8, 2, 128, None])
    for mixed in (0, 1):
        for n in (0, 31, 33, 64, -32, 2 ** 31 - 1):
            assert call(sections=ints(n), mixed=mixed) == -1, n
        assert call(sections=ints(32), mixed=mixed) == 0
        assert call(mixed=mixed) == 0


def test_norm_rope_bwd_refusals(lib):
    names = ["gq", "gk", "q", "k", "qs", "ks"] + HOW + ["dq", "dk", "dqs", "dks", "dqw", "dkw", "total", "hq",
                                                       "hkv", "d", "ws", "wsb", "stream"]
    call = refusals(lib.attn_qk_norm_rope_bwd, names,
                    [None, FAKE, FAKE, FAKE, 1536, 1536] + HOW_GOOD
                    + [FAKE, FAKE, 1024, 256, FAKE, FAKE, 5, 8, 2, 128, FAKE, 1 << 20, None])
    assert call() == -1                          # no dq_out
    for bad in (dict(dq=None), dict(dk=P(4104)), dict(dqs=1000), dict(dks=252), dict(gk=None), dict(dqw=None),
                dict(dkw=P(4097)), dict(qw=None), dict(kw=None)):
        assert call(gq=FAKE, **bad) == -1, bad
    for bad in (dict(ws=None), dict(wsb=16), dict(ws=P(4096 + 16))):
        assert call(gq=FAKE, **bad) == -3, bad
    norm_rope_refusals(lambda **kw: call(**({"dqw": None, "dkw": None} if kw.get("total") == 0 else {}), **kw))
    assert binding.load().attn_qk_norm_rope_bwd_workspace_bytes(128) == 304 * 128 * 4
    assert binding.load().attn_qk_norm_rope_bwd_workspace_bytes(96) == 0


def test_append_refusals(lib):
    names = ["q", "k", "v", "qs", "ks", "vs"] + HOW + ["qo", "kc", "vc", "slots", "total", "hq", "hkv", "d", "ps",
                                                      "np", "stream"]
    call = refusals(lib.attn_kvcache_append_norm_rope, names,
                    [FAKE, FAKE, None, 1536, 1536, 1536] + HOW_GOOD
                    + [FAKE] * 4 + [5, 8, 2, 128, 16, 9, None])
    norm_rope_refusals(call)
    assert call() == -1                          # no v
    for bad in (dict(v=P(4104)), dict(vs=8), dict(qo=None), dict(kc=None), dict(vc=P(4104)), dict(slots=None),
                dict(slots=P(4098)), dict(ps=0), dict(np=0)):
        assert call(**{"v": FAKE, **bad}) == -1, bad
    assert call(v=FAKE, np=1 << 27) == -2        # cache rows past 31 bits


def test_shared_refusals(lib):
    names = ["q", "kc", "vc", "sl", "bt", "gs", "pl", "cu", "ps", "out", "lse", "batch", "groups", "total", "mq",
             "hq", "hkv", "d", "mp", "np", "scale", "ws", "wsb", "stream"]
    call = refusals(lib.attn_decode_kvcache_shared, names,
                    [FAKE] * 7 + [None, 64, FAKE, FAKE, 2, 1, 2, 1, 8, 2, 128, 4, 16, 0.1, FAKE, 1 << 30, None])
    for bad in (dict(q=None), dict(kc=P(4104)), dict(vc=None), dict(sl=None), dict(bt=P(4097)), dict(gs=None),
                dict(pl=None), dict(out=P(4104)), dict(lse=None), dict(lse=P(4098)), dict(cu=P(4097)), dict(batch=-1),
                dict(groups=-1), dict(total=-1), dict(mq=-1), dict(hq=3), dict(hkv=0), dict(mp=0), dict(np=0),
                dict(ps=0), dict(total=3), dict(scale=0.0), dict(scale=float("nan")), dict(scale=-1.0)):
        assert call(**bad) == -1, bad
    for bad in (dict(d=96), dict(ps=48), dict(ps=8), dict(ps=192), dict(batch=70000, total=70000), dict(hq=258),
                dict(groups=70000), dict(np=1 << 30), dict(mp=1 << 25), dict(total=1 << 28, cu=FAKE)):
        assert call(**bad) == -2, bad
    for bad in (dict(ws=None), dict(wsb=16), dict(ws=P(4096 + 16))):
        assert call(**bad) == -3, bad
    assert call(batch=0, total=0) == 0
    assert call(total=0, cu=FAKE) == 0
    need = binding.attn_decode_kvcache_shared_workspace_bytes
    assert need(64, 1, 64, 32, 8, 128) < 40 << 20
    assert need(2, 1, 2, 7, 2, 64) == 0
    assert need(2, 1, 2, 8, 2, 96) == 0


def test_binding_refuses_cpu_tensors(lib):
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    x = lambda *s: torch.zeros(s, dtype=BF16)  # noqa: E731
    with pytest.raises(ValueError):
        binding.attn_kvcache_plan(i(2), i(2), i(2, 4), i(8), i(1), 16, 16, 5)
    with pytest.raises(ValueError):
        binding.attn_qk_norm_rope(x(3, 4, 64), x(3, 2, 64))
    with pytest.raises(ValueError):
        binding.attn_qk_norm_rope_bwd(x(3, 4, 64), x(3, 2, 64), x(3, 4, 64), x(3, 2, 64))
    with pytest.raises(ValueError):
        binding.attn_kvcache_append_norm_rope(x(3, 4, 64), x(3, 2, 64), x(3, 2, 64), x(2, 16, 2, 64),
                                              x(2, 16, 2, 64), i(3))
    with pytest.raises(ValueError):
        binding.attn_decode_kvcache_shared(x(2, 4, 64), x(2, 16, 2, 64), x(2, 16, 2, 64), i(2), i(2, 4))
    with pytest.raises(TypeError):
        binding.attn_qk_norm_rope(None, None)


def test_the_package_offers_the_calls():
    import exact_attention_70_gb300 as attn
    for name in ("attn_kvcache_plan", "attn_qk_norm_rope", "attn_qk_norm_rope_bwd",
                 "attn_kvcache_append_norm_rope", "attn_decode_kvcache_shared"):
        assert name in attn.__all__ and getattr(attn, name) is getattr(binding, name)
