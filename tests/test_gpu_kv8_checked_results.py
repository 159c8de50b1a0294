"""The bounds-checking debug build on the 8-bit cache's four calls: silent on valid inputs, the bytes and
values that it writes those of the definition, and every output the regular build's bit for bit."""
import pytest
import torch

from exact_attention_70_gb300 import binding
from exact_attention_70_gb300 import build as attn_build
from tests import kv8_exact
from tests.kv8_exact import kv8_case
from tests.test_gpu_checked_build import checked  # noqa: F401
from tests.test_gpu_kv8 import append, chunk, dev, gpu_cache
from tests.test_gpu_kv8_range import far_rows, reference, same_stored

pytestmark = pytest.mark.gpu

CASES = [  # new tokens, heads, d, rotary, window, rows far apart
    ([3, 1], 24, 64, 64, (-1, -1), False),         # the 16-row kernel
    ([5, 2], 24, 128, 0, (40, 0), True),
    ([200, 91], 24, 64, 64, (100, 0), False),      # staged: queries in two parts, in one, scales by row
    ([200, 91], 24, 128, 0, (-1, -1), False),
    ([200, 91], 24, 128, 48, (-1, -1), True),
]


def case(i):
    new, heads, d, rotary, window, far = CASES[i]
    c = kv8_case([300, 41], new, heads, 3, d, 32, seed=480 + i, rotary_dim=rotary, spread=0.5, padding=2)
    if far:
        far_rows(c, d, 480 + i)
    return c, window


def run(i):
    """Every output of the calls as a server makes them."""
    c, window = case(i)
    alone = gpu_cache(c)
    append(binding, c, alone)
    cache = gpu_cache(c)
    out, lse = (torch.zeros(s, dtype=t, device="cuda") for s, t in
                ((c.q.shape, torch.bfloat16), ((c.q.shape[1], c.q.shape[0]), torch.float32)))
    chunk(binding, c, cache, True, window, out=out, lse=lse)
    lens = [a + b for a, b in zip(c.ctx, c.new)]
    sl, bt = dev(torch.tensor(lens, dtype=torch.int32)), dev(c.block_table)
    one = binding.attn_decode_kvcache_fp8(dev(c.q[:2]), *cache, sl, bt)
    cu = dev(torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32))
    kv = binding.attn_kvcache_read_fp8(*cache, bt, cu, sum(lens))
    torch.cuda.synchronize()
    assert binding.attn_get_device_status() == 0
    return [t.cpu() for t in (*alone, *cache, out, lse, *one, *kv)]


@pytest.fixture(scope="module")
def results(request):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    attn_build.build()
    binding.load()
    regular = [run(i) for i in range(len(CASES))]
    request.getfixturevalue("checked")
    return regular, [run(i) for i in range(len(CASES))]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_checked_build_gives_the_regular_results(results, i):
    for a, b in zip(results[0][i], results[1][i]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("i", range(len(CASES)))
def test_checked_build_gives_the_defined_results(results, i):
    c, window = case(i)
    got = results[1][i]
    arrays = kv8_exact.appended(c)
    same_stored(got[:4], arrays)
    same_stored(got[4:8], arrays)
    T = sum(c.new)
    kv8_exact.check(got[8][:T], got[9][:, :T].t(), reference(c, arrays, True, window), 2.0 ** -11,
                    c.rotary_cos is not None)
    c.ctx, c.new, c.q = [a + b for a, b in zip(c.ctx, c.new)], [0, 0], c.q[:2]
    kv8_exact.check(got[10], got[11], reference(c, arrays), 2.0 ** -11, False)
    rows = [kv8_exact.read_back(arrays, c.block_table.numpy(), b, n, c.page_size) for b, n in enumerate(c.ctx)]
    for j in (0, 1):
        want = torch.cat([torch.from_numpy(r[j]) for r in rows])
        assert torch.equal(got[12 + j].double(), want)
