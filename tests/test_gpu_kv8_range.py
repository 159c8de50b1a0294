"""The calls on the 8-bit paged KV cache over the whole range of what it stores and of what a mask
leaves out, against the fp64 definition (tests.kv8_exact): rows of zeros, keys and values from
2^-126 to 2^127, values far apart within a sequence, large, infinite and NaN values that no row sees,
pages that a window has left behind.

The bounds are those of kv8_exact.check: a logit is off by dS d 2^-23 for its fp32 sums of d products
(and dS 2^-20 where the query was rotated and goes to the tensor cores as two f16 numbers of 11 bits
each), a weight by 2^-11 as an f16 operand (below f16's normal range as reference() says) and by 2^-20
for exp2 and the division, O by 2^-8 as bf16."""
import numpy as np
import pytest
import torch

from tests import kv8_exact
from tests.kv8_exact import kv8_case
from tests.test_gpu_kv8 import append, attn, chunk, decode, dev, gpu_cache  # noqa: F401

pytestmark = pytest.mark.gpu

SHORT, LONG = [3, 5], [200, 90]  # new tokens: on the codes; staged (32:8 heads)
EXPONENTS = [-124, -110, -90, 60, 80, 100, 108, 116, 124]
BIG = [2.0 ** 26, 2.0 ** 40, 2.0 ** 90, 3.3e38]


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


def same_stored(cache, arrays):
    """The same bytes, but for the sign of zeros (a sum of two zeros has none)."""
    for i, (got, want) in enumerate(zip(cache, arrays)):
        got = got.cpu().numpy()
        assert np.array_equal(*(np.where(x == 0x80, 0, x) if i < 2 else x for x in (got, want)))


def reference(c, arrays, causal=True, window=(-1, -1)):
    """kv8_exact.attention of c's tokens, dS over the keys that a row sees, and W with what f16 weights
    lose below their normal range, 2^-14: 2^-25 a weight.  Either the largest weight times its value's scale,
    P_j 2^e_j, is brought to 2 or above: this is then 2^-26 of it a code; or, where no scales are more than
    2^22 apart, the largest weight is brought to 2^7: 2^-32 of |v_j|.  (check() takes 2^-11 of W.)"""
    decode = not any(c.new)
    new = [1] * len(c.ctx) if decode else c.new
    T = sum(new)
    O, LSE, dS, W = [x[:T] for x in kv8_exact.attention(c, arrays, causal, window)]
    g = O.shape[1] // c.k_cache.shape[2]
    table, t0 = c.block_table.numpy(), 0
    for b, n in enumerate(new):
        L = c.ctx[b] + (0 if decode else n)
        pos = L - n + np.arange(n)
        q = c.q[t0:t0 + n].double().numpy()
        if not decode:
            q = kv8_exact.rotate(q, pos, c.rotary_cos, c.rotary_sin, c.interleaved)
        k, v = kv8_exact.read_back(arrays, table, b, L, c.page_size)
        j = np.arange(L)
        e = arrays[3][table[b, j // c.page_size], :, j % c.page_size].astype(np.float64) - 127
        right = 0 if causal else window[1]
        seen = np.ones((n, L), bool) if right < 0 else j <= pos[:, None] + right
        if window[0] >= 0:
            seen &= j >= pos[:, None] - window[0]
        for h in range(O.shape[1] if L else 0):
            kh, vh, eh = k[:, h // g], np.abs(v[:, h // g]), np.exp2(e[:, h // g])
            dS[t0:t0 + n, h] = c.scale * np.where(seen, np.abs(q[:, h]) @ np.abs(kh).T, 0.0).max(1)
            s = np.where(seen, c.scale * (q[:, h] @ kh.T), -np.inf)
            top = (np.exp(s - np.maximum(s.max(1), -1e300)[:, None]) * eh).max(1)
            # (rows of the smallest scale, zeros, do not count among the scales)
            near = np.minimum(eh, 2.0 ** 22 * eh.min(initial=np.inf, where=eh > 2.0 ** -126))
            W[t0:t0 + n, h] += seen @ (vh / eh[:, None] * near[:, None]) * 2.0 ** -21
            W[t0:t0 + n, h] += top[:, None] * (seen @ (vh / eh[:, None])) * 2.0 ** -15
        t0 += n
    return O, LSE, dS, W


def check_chunk(attn, c, causal=True, window=(-1, -1), what="", **kw):  # noqa: F811
    cache = gpu_cache(c)
    out, lse = chunk(attn, c, cache, causal, window, **kw)
    assert attn.attn_get_device_status() == 0, what
    arrays = kv8_exact.appended(c)
    same_stored(cache, arrays)
    T = sum(c.new)
    kv8_exact.check(out[:T], lse[:, :T].t(), reference(c, arrays, causal, window), 2.0 ** -11,
                    c.rotary_cos is not None, what)


def check_decode(attn, c, what=""):  # noqa: F811
    out, lse = decode(attn, c)
    kv8_exact.check(out, lse, reference(c, [t.numpy() for t in c.cache]), 2.0 ** -11, False, what)


@pytest.mark.parametrize("rotary", [0, 64])
@pytest.mark.parametrize("window", [(-1, -1), (40, 0)])
@pytest.mark.parametrize("new", [SHORT, LONG])
def test_chunk_of_zero_and_tiny_keys_and_queries(attn, new, window, rotary):  # noqa: F811
    """Logits of 0: uniform weights over what a row sees, whatever the units of its parts."""
    c = kv8_case([70, 30], new, 32, 8, 64, 32, seed=400, rotary_dim=rotary, spread=0.5)
    for b in (0, 1):
        n = c.ctx[b]
        k = np.zeros((n, 8, 64))
        k[:, 4:6] = 2.0 ** -100 * np.random.default_rng(b).standard_normal((n, 2, 64))
        k[:, 6:] = 2.0 ** -13 * np.random.default_rng(b).standard_normal((n, 2, 64))
        put_cached(c, b, np.arange(n), k=k)
    c.k_new[:, :4] = 0
    c.k_new[:, 4:6] *= 2.0 ** -100
    c.k_new[:, 6:] *= 2.0 ** -13
    c.q[:, 0::4] = 0                 # query heads 0 of every kv head, ...
    c.q[:, 1::4] *= 2.0 ** -10
    c.q[:, 2::4] *= 2.0 ** -120
    check_chunk(attn, c, True, window)


def test_calls_on_all_zero_tensors(attn):  # noqa: F811
    """What a program warms up with."""
    for new in (SHORT, LONG):
        c = kv8_case([0, 0], new, 32, 8, 128, 64, seed=401, rotary_dim=128)
        for t in (c.q, c.k_new, c.v_new):
            t.zero_()
        check_chunk(attn, c)
    c = kv8_case([33, 1], None, 4, 2, 64, 16, seed=402)
    c.q.zero_()
    for b, n in enumerate(c.ctx):
        put_cached(c, b, np.arange(n), k=np.zeros((n, 2, 64)), v=np.zeros((n, 2, 64)))
    check_decode(attn, c)


@pytest.mark.parametrize("new", [None, SHORT, LONG])
@pytest.mark.parametrize("scale", [1.2e-38, 1e-20])
def test_softmax_scales_at_the_bottom_of_their_range(attn, scale, new):  # noqa: F811
    """Tiny queries times the smallest scales: logits of 0 to fp32, masked ones still -infinity."""
    c = kv8_case([70, 30], new, 32, 8, 64, 32, seed=403, scale=scale)
    c.q *= 2.0 ** -120
    if new is None:
        check_decode(attn, c)
    else:
        check_chunk(attn, c, True, (40, 0))


def sized(shape, e, aligned, rng):
    """Rows of size 2^e: of any sign, or all positive, whose products with each other add up."""
    return (rng.uniform(1, 2, shape) if aligned else rng.standard_normal(shape)) * 2.0 ** e


@pytest.mark.parametrize("aligned", [False, True])
@pytest.mark.parametrize("e", EXPONENTS)
def test_decode_over_keys_of_any_size(attn, e, aligned):  # noqa: F811
    """Keys of size 2^e and queries of 2^-e: moderate logits."""
    c = kv8_case([300, 40], None, 8, 2, 128, 64, seed=410)
    rng = np.random.default_rng(410)
    for b, n in enumerate(c.ctx):
        put_cached(c, b, np.arange(n), k=sized((n, 2, 128), e, aligned, rng))
    c.q = bf16(sized(c.q.shape, -e, aligned, rng))
    check_decode(attn, c, f"2^{e}")


@pytest.mark.parametrize("aligned", [False, True])
@pytest.mark.parametrize("rotary", [0, 128])
@pytest.mark.parametrize("e", EXPONENTS)
@pytest.mark.parametrize("new", [SHORT, LONG])
def test_chunk_over_keys_of_any_size(attn, new, e, rotary, aligned):  # noqa: F811
    c = kv8_case([200, 40], new, 32, 8, 128, 64, seed=411, rotary_dim=rotary)
    rng = np.random.default_rng(411)
    for b, n in enumerate(c.ctx):
        put_cached(c, b, np.arange(n), k=sized((n, 8, 128), e, aligned, rng))
    c.k_new = bf16(sized(c.k_new.shape, e, aligned, rng))
    c.q = bf16(sized(c.q.shape, -e, aligned, rng))
    check_chunk(attn, c, what=f"2^{e}")


@pytest.mark.parametrize("new", [None, SHORT, LONG])
def test_keys_of_all_sizes_in_one_sequence(attn, new):  # noqa: F811
    """Keys 2^28 apart whose logits are alike: each meets the query in one component, where the query is
    as much smaller; what is left of the keys' rows is larger by 2^7 and meets a zero."""
    n, d = 190, 64
    e = 4.0 * np.arange(8) - 14
    rng = np.random.default_rng(9)

    def keys(i):
        k = np.zeros((len(i), 8, d))
        k[np.arange(len(i)), :, i % 8] = rng.uniform(-2, 2, (len(i), 8)) * 2.0 ** e[i % 8, None]
        k[:, :, 63] = 2.0 ** (e[i % 8, None] + 7)
        return k

    c = kv8_case([n, n], new, 32, 8, d, 32, seed=412, scale=1.0)
    q = np.zeros(c.q.shape)
    q[..., :8] = rng.choice([-1.0, 1.0], q[..., :8].shape) * 2.0 ** -e
    c.q = bf16(q)
    for b in (0, 1):
        put_cached(c, b, np.arange(n), k=keys(rng.permutation(n)))
    if new is None:
        check_decode(attn, c)
    else:
        c.k_new = bf16(keys(rng.permutation(sum(new))))
        check_chunk(attn, c)


@pytest.mark.parametrize("rotary", [0, 64])
@pytest.mark.parametrize("big", BIG)
@pytest.mark.parametrize("new", [[9, 5], LONG])
def test_chunk_beside_large_values_that_rows_do_not_see(attn, new, big, rotary):  # noqa: F811
    """The last new token's value is large, and so is one in the middle: rows before them do not see
    them.  So is a cached one that the window of later rows leaves out."""
    c = kv8_case([90, 130], new, 32, 8, 64, 32, seed=420, rotary_dim=rotary, spread=0.5)
    for b in (0, 1):
        r = new_rows(c, b)
        c.v_new[r.stop - 1, :4] = bf16(c.v_new[r.stop - 1, :4].double() * (big / 8))
        c.v_new[(r.start + r.stop) // 2, 5] = bf16(c.v_new[(r.start + r.stop) // 2, 5].double() * (big / 8))
        put_cached(c, b, [c.ctx[b] - 30], v=np.random.default_rng(b).uniform(-1, 1, (1, 8, 64)) * big)
    check_chunk(attn, c, True, (31, 0), f"{big}")
    check_chunk(attn, c, True, (-1, -1), f"{big}")


@pytest.mark.parametrize("big", BIG)
@pytest.mark.parametrize("new", [[9, 5], LONG])
def test_chunk_beside_large_keys_that_rows_do_not_see(attn, new, big):  # noqa: F811
    c = kv8_case([90, 130], new, 32, 8, 64, 32, seed=421, spread=0.5)
    for b in (0, 1):
        put_cached(c, b, [c.ctx[b] - 30], k=np.random.default_rng(b).uniform(-1, 1, (1, 8, 64)) * big)
    # rows from the third on do not see it; the ones before have queries that keep the logits moderate
    for b in (0, 1):
        r = new_rows(c, b)
        c.q[r.start:r.start + 3] = bf16(c.q[r.start:r.start + 3].double() / big)
    check_chunk(attn, c, True, (31, 0), f"{big}")


@pytest.mark.parametrize("far", [26, 40, 60, 100])
@pytest.mark.parametrize("new", [None, [9, 5], LONG])
def test_large_values_of_small_weight(attn, new, far):  # noqa: F811
    """A value 2^far times the others' whose weight is 2^-(far + 30): the others make the result."""
    d = 64
    c = kv8_case([150, 300], new, 32, 8, d, 32, seed=422, spread=0.0, scale=1.0)
    # component 0 of q is 1 and of the keys 0, but for the far ones' -(far + 30) ln 2
    c.q = bf16(c.q.double() * 2.0 ** -4)
    c.q[..., 0] = 1
    c.k_new[..., 0] = 0
    rng = np.random.default_rng(5)
    for b, n in enumerate(c.ctx):
        k, v = rng.standard_normal((2, n, 8, d))
        k[..., 0] = 0
        at = [0, 41, n - 2]
        k[at], v[at] = 0, v[at] * 2.0 ** far
        k[at, :, 0] = -(far + 30) * np.log(2)
        put_cached(c, b, np.arange(n), k=k, v=v)
    if new is None:
        check_decode(attn, c, f"{far}")
    else:
        check_chunk(attn, c, what=f"{far}")


@pytest.mark.parametrize("new", [None, [9, 5], LONG])
def test_large_values_first_then_larger_logits(attn, new):  # noqa: F811
    """A large value that carried all the weight until keys came whose logits are far above its own."""
    d = 64
    c = kv8_case([600, 300], new, 32, 8, d, 32, seed=423, spread=0.0, scale=1.0)
    c.q = bf16(c.q.double() * 2.0 ** -4)
    c.q[..., 0] = 1
    c.k_new[..., 0] = 70
    rng = np.random.default_rng(6)
    for b, n in enumerate(c.ctx):
        k, v = rng.standard_normal((2, n, 8, d))
        k[..., 0] = np.where(np.arange(n) < 100, 0.0, 70.0)[:, None]
        v[:100] *= 2.0 ** 60
        put_cached(c, b, np.arange(n), k=k, v=v)
    if new is None:
        check_decode(attn, c)
    else:
        check_chunk(attn, c)


def far_rows(c, d, seed):
    """Rows of kv head 1, cached and new, 2^40 apart; its queries small enough for moderate logits."""
    rng = np.random.default_rng(seed)
    for b, n in enumerate(c.ctx):
        if n:
            k, v = (rng.standard_normal((n, 3, d)) for _ in "kv")
            for x in (k, v):
                x[:, 1] *= 2.0 ** rng.uniform(-20, 20, (n, 1))
            put_cached(c, b, np.arange(n), k=k, v=v)
    f = torch.from_numpy(2.0 ** rng.uniform(-20, 20, (2, c.k_new.shape[0], 1)))
    c.k_new[:, 1], c.v_new[:, 1] = bf16(c.k_new[:, 1].double() * f[0]), bf16(c.v_new[:, 1].double() * f[1])
    g = c.q.shape[1] // 3
    c.q[:, g:2 * g] *= 2.0 ** -18


@pytest.mark.parametrize("causal,window", [(True, (-1, -1)), (True, (100, 0)), (False, (30, 7)),
                                           (False, (-1, -1))])
@pytest.mark.parametrize("d,rotary", [(64, 0), (64, 64), (128, 0), (128, 48)])
def test_chunk_whose_rows_are_far_apart(attn, d, rotary, causal, window):  # noqa: F811
    """Staged, one of three kv heads: its neighbours take their usual way, an odd number of keys in all,
    a sequence without cached tokens, one without new ones."""
    c = kv8_case([301, 0, 77, 5], [200, 131, 0, 65], 24, 3, d, 32, seed=425, rotary_dim=rotary)
    far_rows(c, d, 425)
    check_chunk(attn, c, causal, window)


@pytest.mark.parametrize("rotary", [0, 128])
def test_graph_replayed_as_rows_move_apart(attn, rotary):  # noqa: F811
    """A captured chunk whose rows lie close, replayed with rows far apart and with close ones again."""
    near, far = (kv8_case([301, 77], [200, 65], 24, 3, 128, 32, seed=426, rotary_dim=rotary) for _ in "ab")
    far_rows(far, 128, 426)

    def inputs(c):
        return [c.q, c.k_new, c.v_new, *c.cache]

    held = [t.cuda() for t in inputs(near)]
    rest = [dev(t) for t in (near.cache_seqlens, near.block_table, near.cu_seqlens_q)]
    tables = [dev(near.rotary_cos), dev(near.rotary_sin)]

    def step():
        return attn.attn_fwd_kvcache_fp8(*held, *rest, 200, 643, near.scale, True, -1, -1, *tables)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for c in (far, near, far):
        for h, t in zip(held, inputs(c)):
            h.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        kv8_exact.check(outs[0], outs[1].t(), reference(c, kv8_exact.appended(c)), 2.0 ** -11, rotary > 0)
        got = [t.clone() for t in outs]
        for h, t in zip(held, inputs(c)):
            h.copy_(t)
        assert all(torch.equal(a, b) for a, b in zip(got, step()))
    assert attn.attn_get_device_status() == 0


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("rotary", [0, 128])
def test_what_follows_a_chunk_finds_it_finished(attn, rotary, far):  # noqa: F811
    """Kernels right behind the call on its stream, and the same call on two streams at once."""
    cases = [kv8_case([3000, 701], [900, 333], 24, 3, 128, 64, seed=427 + i, rotary_dim=rotary) for i in (0, 1)]
    for i, c in enumerate(cases):
        if far:
            far_rows(c, 128, 427 + i)
    caches = [gpu_cache(c) for c in cases]
    ins = [([dev(t) for t in (c.q, c.k_new, c.v_new)],
            [dev(t) for t in (c.cache_seqlens, c.block_table, c.cu_seqlens_q)],
            [dev(c.rotary_cos), dev(c.rotary_sin)]) for c in cases]

    def call(i, out, lse, stream=None):
        a, b, r = ins[i]
        return attn.attn_fwd_kvcache_fp8(*a, *caches[i], *b, 900, 4934, cases[i].scale, True, -1, -1, *r, out=out,
                                         lse=lse, stream=stream)

    outs = [(torch.empty_like(x[0][0]), torch.empty(24, 1233, device="cuda")) for x in ins]
    want = [[t.clone() for t in call(i, *o)] for i, o in enumerate(outs)]
    torch.cuda.synchronize()
    c = cases[0]
    kv8_exact.check(want[0][0], want[0][1].t(), reference(c, kv8_exact.appended(c)), 2.0 ** -11, rotary > 0)
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                for t in outs[i]:
                    t.fill_(7)
                call(i, *outs[i], stream=s)
                got[i].append([t.clone() for t in outs[i]])
    torch.cuda.synchronize()
    assert attn.attn_get_device_status() == 0
    for i in (0, 1):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


@pytest.mark.parametrize("new", [None, SHORT, LONG])
@pytest.mark.parametrize("e", [-60, -100, -120])
def test_tiny_values(attn, e, new):  # noqa: F811
    """Values down to bf16's smallest: O is as exact as its type holds it."""
    c = kv8_case([150, 300], new, 32, 8, 64, 32, seed=424)
    rng = np.random.default_rng(7)
    for b, n in enumerate(c.ctx):
        put_cached(c, b, np.arange(n), v=rng.standard_normal((n, 8, 64)) * 2.0 ** e)
    c.v_new = bf16(c.v_new.double() * 2.0 ** e)
    out, lse = decode(attn, c) if new is None else chunk(attn, c, gpu_cache(c))
    O, LSE, dS, W = reference(c, [t.numpy() for t in c.cache] if new is None else kv8_exact.appended(c))
    # (2^e taken out: bf16 values below 2^-126 are spaced 2^-133, which 2^(-133 - e) adds)
    out = out.double().cpu().numpy() * 2.0 ** -e
    err = np.abs(out - O * 2.0 ** -e)
    x = dS * 64 * 2.0 ** -23
    bound = 2.0 ** -8 * np.abs(O) * 2.0 ** -e + (1 + 2.0 ** -8) * (
        np.expm1(2 * x) + 2.0 ** -11 + 2.0 ** -20)[..., None] * W * 2.0 ** -e + 2.0 ** (-133 - e)
    assert np.all(err <= bound), (err / bound).max()


@pytest.mark.parametrize("rotary", [0, 64])
@pytest.mark.parametrize("new", [SHORT, LONG])
def test_nothing_before_the_window_is_looked_at(attn, new, rotary):  # noqa: F811
    """Pages that end before the first key that a new token sees are given up (-1 in the table), and
    the slots of its own page before it hold NaN."""
    window = 70
    c = kv8_case([1000, 333], new, 32, 8, 64, 16, seed=430, rotary_dim=rotary, spread=0.5)
    for b, n in enumerate(c.ctx):
        first = n - window
        c.block_table[b, :first // 16] = -1
        page = int(c.block_table[b, first // 16])
        for t in (c.k_cache, c.v_cache):
            t[page, :first % 16] = 0x7F
        for t in (c.k_scale, c.v_scale):
            t[page, :, :first % 16] = 255
    cache = gpu_cache(c)
    out, lse = chunk(attn, c, cache, True, (window, 0))
    assert attn.attn_get_device_status() == 0
    # the same with everything before the window in order
    good = kv8_case([1000, 333], new, 32, 8, 64, 16, seed=430, rotary_dim=rotary, spread=0.5)
    ref = reference(good, kv8_exact.appended(good), True, (window, 0))
    kv8_exact.check(out, lse.t(), ref, 2.0 ** -11, rotary > 0)


@pytest.mark.parametrize("rotary", [0, 64])
@pytest.mark.parametrize("new", [SHORT, LONG])
def test_rows_that_see_a_nan_key_say_so(attn, new, rotary):  # noqa: F811
    """O and LSE of every row that sees it are NaN: an LSE of -infinity would stand for no keys."""
    c = kv8_case([40, 300], new, 32, 8, 64, 16, seed=440, rotary_dim=rotary, spread=0.5)
    c.k_cache[int(c.block_table[0, 1]), 3, 2, 5] = 0x7F      # kv head 2 of sequence 0
    c.v_scale[int(c.block_table[1, 0]), 5, 2] = 255          # kv head 5 of sequence 1
    cache = gpu_cache(c)
    out, lse = chunk(attn, c, cache)
    arrays = kv8_exact.appended(c)
    same_stored(cache, arrays)
    a, b = new_rows(c, 0), new_rows(c, 1)
    assert torch.isnan(out[a, 8:12]).all() and torch.isnan(lse[8:12, a]).all()
    assert torch.isnan(out[b, 20:24]).all()                  # a NaN value: O alone
    assert torch.isfinite(lse[20:24, b]).all()
    ref = reference(c, arrays)
    for rows, heads in ((a, slice(0, 8)), (a, slice(12, 32)), (b, slice(0, 20)), (b, slice(24, 32))):
        kv8_exact.check(out[rows, heads], lse[heads, rows].t(), [x[rows, heads] for x in ref], 2.0 ** -11,
                        rotary > 0)


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


@pytest.mark.parametrize("e", [-132, -126, -118, 118, 126])
@pytest.mark.parametrize("new", [SHORT, LONG])
def test_rotated_queries_of_any_size(attn, new, e):  # noqa: F811
    """Queries of 2^e on keys of 2^-e (as far as their type goes), the scale making up for the rest."""
    k = max(-e, -118) if e > 0 else min(-e, 120)
    c = kv8_case([100, 40], new, 32, 8, 64, 32, seed=460, rotary_dim=64, scale=2.0 ** -(e + k) / 8)
    top = float(torch.finfo(torch.bfloat16).max)
    for b, n in enumerate(c.ctx):
        put_cached(c, b, np.arange(n), k=np.random.default_rng(b).standard_normal((n, 8, 64)) * 2.0 ** k)
    c.k_new = bf16(c.k_new.double() * 2.0 ** k)
    c.q = bf16(np.clip(c.q.double().numpy() * 2.0 ** e, -top, top))
    cache = gpu_cache(c)
    out, lse = chunk(attn, c, cache)
    assert attn.attn_get_device_status() == 0
    arrays = kv8_exact.appended(c)
    same_stored(cache, arrays)
    O, LSE, dS, W = reference(c, arrays)
    # A query's elements have a floor: f16 numbers are 2^-24 apart below 2^-14 and a unit of them is
    # 2^-120 at least, so an element is off by up to 2^-145, and a logit by scale sum_d |k_d| 2^-145
    # more; check() takes dS 2^-20 for the rotation, so it joins dS times 2^20.
    g = O.shape[1] // 8
    for b, n in enumerate(c.new):
        k = np.abs(kv8_exact.read_back(arrays, c.block_table.numpy(), b, c.ctx[b] + n, 32)[0]).sum(-1).max(0)
        dS[new_rows(c, b)] += c.scale * np.repeat(k, g) * 2.0 ** -145 * 2.0 ** 20
    kv8_exact.check(out, lse.t(), (O, LSE, dS, W), 2.0 ** -11, True, f"2^{e}")


def test_max_seqlen_q_far_above_the_tokens_of_the_call(attn):  # noqa: F811
    """No sequence has more new tokens than the call: any larger bound gives the same results."""
    for new in (SHORT, LONG):
        c = kv8_case([70, 30], new, 32, 8, 64, 32, seed=470, rotary_dim=64)
        want = chunk(attn, c, gpu_cache(c))
        args = [dev(t) for t in (c.q, c.k_new, c.v_new)]
        rest = [dev(t) for t in (c.cache_seqlens, c.block_table, c.cu_seqlens_q)]
        for bound in (sum(new), 10 ** 6, 2 ** 31 - 1):
            got = attn.attn_fwd_kvcache_fp8(*args, *gpu_cache(c), *rest, bound, 100 + sum(new), c.scale, True,
                                            -1, -1, dev(c.rotary_cos), dev(c.rotary_sin))
            torch.cuda.synchronize()
            assert attn.attn_get_device_status() == 0
            for g, w in zip(got, want):
                assert torch.allclose(g.float(), w.float(), rtol=2.0 ** -7, atol=2.0 ** -7)
