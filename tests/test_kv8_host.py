"""CPU checks of the 8-bit KV cache: its fp64 definition in tests.kv8_exact against the oracle's
e4m3 codec and by hand, and what the C ABI and the binding refuse before touching a device."""
import ctypes

import numpy as np
import pytest
import torch

from exact_attention_70_gb300 import binding
from exact_attention_70_gb300 import build as attn_build
from oracle import oracle
from tests import kv8_exact

P = ctypes.c_void_p
FAKE = P(4096)  # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def lib():
    attn_build.build()
    return binding.load()


def test_grid_is_the_e4m3_format():
    assert np.array_equal(kv8_exact.GRID, oracle.e4m3_to_f64(np.arange(127)))
    assert np.array_equal(kv8_exact.VALUES[128:255], -kv8_exact.GRID)
    assert kv8_exact.GRID[-1] == 448.0 and np.isnan(kv8_exact.VALUES[[127, 255]]).all()


def test_quantised_rows_by_hand():
    x = np.zeros((7, 4))
    x[0] = [448, -448, 1, 0.5]            # e = 0
    x[1] = [448.1, 16, 0, -17]            # just above: e = 1, 17 / 2 ties between 8 and 9 -> 8
    x[2] = [2.0 ** -130, 0, 0, 0]         # below the smallest scale: e = -126, a subnormal code
    x[4] = [np.inf, 2, -np.nan, -np.inf]  # non-finite elements: the NaN code, not in the maximum
    x[5] = [3.3e38, -1e38, 0, 0]
    x[6] = [1.0, 1.0625, 1.1875, 2.0 ** -30]
    codes, b = kv8_exact.quantise_rows(x)
    assert list(b) == [127, 128, 1, 1, 127 - 7, 127 + 120, 127 - 8]
    v = kv8_exact.VALUES[codes] * np.exp2(b.astype(float) - 127)[:, None]
    assert list(v[0]) == [448, -448, 1, 0.5]
    assert list(v[1]) == [448, 16, 0, -16]
    assert v[2][0] == 2.0 ** -130 and codes[2][0] == 24
    assert not codes[3].any()
    assert list(codes[4][[0, 2, 3]]) == [0x7F] * 3 and v[4][1] == 2
    assert list(v[6]) == [1.0, 1.0, 1.25, 0.0]  # ties to the even code


def test_quantised_rows_match_the_oracles_codec():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((40, 64)) * np.exp2(rng.uniform(-30, 30, (40, 1)))
    codes, b = kv8_exact.quantise_rows(x)
    for i in range(40):
        e = float(b[i]) - 127
        top = np.abs(x[i]).max()
        assert top <= 448 * 2 ** e and top > 448 * 2 ** (e - 1)
        assert [oracle.f64_to_e4m3(y) for y in x[i] * 2.0 ** -e] == list(codes[i])


def test_rotation_by_hand():
    cos, sin = torch.tensor([[1.0], [0.0]]), torch.tensor([[0.0], [1.0]])
    x = np.array([[[1.0, 2.0, 3.0]], [[1.0, 2.0, 3.0]]])
    for inter in (False, True):
        assert np.array_equal(kv8_exact.rotate(x, np.array([0, 1]), cos, sin, inter),
                              [[[1, 2, 3]], [[-2, 1, 3]]])


def refusals(f, names, good):
    def call(**kw):
        a = dict(zip(names, good))
        assert set(kw) <= set(a)
        a.update(kw)
        return f(*a.values())
    return call


SIZES = ["batch", "total", "hkv", "d", "ps", "mp", "np"]


def common_refusals(call):
    assert call(d=96) == -2
    assert call(ps=48) == -2                    # neither divides 64 nor is a multiple of it
    assert call(ps=8) == -2
    assert call(ps=0) == -1
    assert call(mp=0) == -1
    assert call(np=0) == -1
    assert call(hkv=0) == -1
    assert call(batch=-1) == -1
    assert call(batch=70000) == -2
    assert call(np=1 << 30) == -2               # cache rows past 31 bits
    assert call(kc=None) == -1
    assert call(vs=None) == -1
    assert call(kc=P(4104)) == -1               # caches and scales are 16-byte aligned
    assert call(ks=P(4104)) == -1
    assert call(bt=P(4097)) == -1
    assert call(batch=0) == 0


def test_append_refusals(lib):
    names = ["k", "v", "kc", "vc", "ks", "vs", "sl", "bt", "cu", "cos", "sin", "rot", "rows", "inter",
             "batch", "total", "hkv", "d", "ps", "mp", "np", "stream"]
    call = refusals(lib.attn_kvcache_append_fp8, names,
                    [FAKE] * 9 + [None, None, 0, 0, 0, 2, 16, 2, 128, 64, 4, 16, None])
    common_refusals(call)
    assert call(total=-1) == -1
    assert call(k=None) == -1
    assert call(v=P(4100)) == -1
    assert call(rot=24, cos=FAKE, sin=FAKE, rows=9) == -2
    assert call(rot=144, cos=FAKE, sin=FAKE, rows=9) == -2   # past the head
    assert call(rot=64) == -1                                # rotary without tables
    assert call(rot=64, cos=FAKE, sin=FAKE, rows=0) == -1
    assert call(rot=64, cos=P(4100), sin=FAKE, rows=9) == -1
    assert call(total=0) == 0


def test_read_refusals(lib):
    names = ["kc", "vc", "ks", "vs", "bt", "cu", "k", "v", "batch", "total", "hkv", "d", "ps", "mp", "np",
             "stream"]
    call = refusals(lib.attn_kvcache_read_fp8, names, [FAKE] * 8 + [2, 16, 2, 128, 64, 4, 16, None])
    common_refusals(call)
    assert call(total=-1) == -1
    assert call(k=None) == -1
    assert call(v=P(4100)) == -1
    assert call(cu=None) == -1
    assert call(total=0) == 0


def test_decode_refusals(lib):
    names = ["q", "kc", "vc", "ks", "vs", "sl", "bt", "ps", "out", "lse", "batch", "hq", "hkv",
             "d", "mp", "np", "scale", "ws", "wsb", "stream"]
    call = refusals(lib.attn_decode_kvcache_fp8, names,
                    [FAKE] * 7 + [64, FAKE, FAKE, 2, 8, 2, 128, 4, 16, 0.1, FAKE, 1 << 24, None])
    common_refusals(call)
    assert call(hq=3) == -1
    for bad in (0.0, -1.0, float("nan"), float("inf"), 1e-39):
        assert call(scale=bad) == -1
    assert call(q=None) == -1
    assert call(out=P(4100)) == -1
    assert call(ws=None) == -3
    assert call(wsb=16) == -3
    assert call(ws=P(4096 + 16)) == -3
    need = binding.attn_decode_kvcache_fp8_workspace_bytes
    # two parts of 16 rows of O and LSE and one entry a CTA; at most two CTAs an SM
    assert need(64, 32, 8, 128, 256, 128) == 304 * (2 * 16 * (128 + 1) * 4 + 16)
    assert need(1, 8, 2, 64, 64, 4) == 2 * 2 * 16 * (64 + 1) * 4 + 256  # 2 chunks, 2 heads
    assert need(2, 8, 2, 96, 64, 4) == 0
    assert need(2, 7, 2, 64, 64, 4) == 0


def test_chunk_refusals(lib):
    names = ["q", "k", "v", "kc", "vc", "ks", "vs", "sl", "bt", "cu", "cos", "sin", "rot", "rows", "inter",
             "out", "lse", "batch", "total", "mq", "mk", "hq", "hkv", "d", "ps", "mp", "np", "scale",
             "causal", "wl", "wr", "ws", "wsb", "stream"]
    call = refusals(lib.attn_fwd_kvcache_fp8, names,
                    [FAKE] * 10 + [None, None, 0, 0, 0, FAKE, FAKE, 2, 16, 8, 64, 8, 2, 128, 64, 4, 16,
                                   0.1, 1, -1, -1, FAKE, 1 << 30, None])
    common_refusals(call)
    assert call(hq=3) == -1
    assert call(mq=-1) == -1
    assert call(mk=-1) == -1
    assert call(wl=-2) == -1
    assert call(scale=0.0) == -1
    assert call(rot=64) == -1
    assert call(q=P(4100)) == -1
    assert call(lse=None) == -1
    assert call(ws=None, rot=128, cos=FAKE, sin=FAKE, rows=99) == -3
    assert call(wsb=16, rot=128, cos=FAKE, sin=FAKE, rows=99) == -3
    assert call(total=0) == 0


def test_more_heads_than_the_kernels_index_are_refused(lib):
    decode = lib.attn_decode_kvcache_fp8
    assert decode(*[FAKE] * 7, 64, FAKE, FAKE, 0, 65535, 1, 128, 4, 16, 0.1, FAKE, 0, None) == 0
    assert decode(*[FAKE] * 7, 64, FAKE, FAKE, 0, 65536, 1, 128, 4, 16, 0.1, FAKE, 0, None) == -2
    chunk = lib.attn_fwd_kvcache_fp8
    for heads, want in ((65535, 0), (65536, -2)):
        assert chunk(*[FAKE] * 10, None, None, 0, 0, 0, FAKE, FAKE, 0, 16, 8, 64, heads, 1, 128, 64, 4, 16,
                     0.1, 1, -1, -1, FAKE, 1 << 30, None) == want


def test_binding_refuses_cpu_tensors_and_wrong_shapes(lib):
    c = kv8_exact.kv8_case([3], [2], 4, 2, 64, 16, seed=1)
    with pytest.raises(ValueError):
        binding.attn_kvcache_append_fp8(c.k_new, c.v_new, *c.cache, c.cache_seqlens, c.block_table,
                                        c.cu_seqlens_q)
    with pytest.raises(ValueError):
        binding.attn_decode_kvcache_fp8(c.q, *c.cache, c.cache_seqlens, c.block_table)
