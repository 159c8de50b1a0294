"""The bounds-checking debug build on the step's calls: silent on valid inputs, and every output the regular
build's bit for bit."""
import pytest
import torch

from exact_attention_70_gb300 import binding
from exact_attention_70_gb300 import build as attn_build
from tests.step_exact import shared_case
from tests.test_gpu_checked_build import checked  # noqa: F401
from tests.test_gpu_norm_rope import case, gpu, how, parts
from tests.test_gpu_plan import ints, make
from tests.test_gpu_shared import call, dev

pytestmark = pytest.mark.gpu

ROPE = [dict(T=65, Hq=32, Hkv=8, d=128, rot=128),
        dict(T=700, Hq=5, Hkv=1, d=64, rot=48, axes=3, sections=(8, 8, 8), inter=True)]
SHARED = [([(300, [(1, 40), (1, 7), (1, None)]), (2000, [(1, i) for i in range(40)])], 8, 2, 128, 64, 0),
          ([(333, [(4, 10), (0, 7), (130, 3)]), (130, [(2, 0), (9, 100)])], 14, 2, 64, 16, 5)]


def run():
    """Every output of the calls."""
    got = []
    for pad, sizes in ((5, ([15, 0, 300], [40, 3, 0])), (0, ([1] * 9, [500] * 9))):
        table, free, count, pages = make(*sizes, 16, seed=3)
        t = ints(table).view(len(table), -1)
        got += [t, *binding.attn_kvcache_plan(ints(sizes[0]), ints(sizes[1]), t, ints(free), ints([count]), 16,
                                              pages, sum(sizes[1]) + pad)]
    for i, kw in enumerate(ROPE):
        c = case(seed=i, **kw)
        q, k, v = parts(c, True)
        cache = torch.zeros((60, 16, c["Hkv"], c["d"]), dtype=torch.bfloat16, device="cuda")
        other = cache.clone()
        slots = torch.randperm(960, generator=torch.Generator().manual_seed(i))[:c["T"]].int().cuda()
        got += [*binding.attn_qk_norm_rope(q, k, **how(c)),
                *binding.attn_qk_norm_rope_bwd(gpu(c["gq"]), gpu(c["gk"]), q, k, **how(c)),
                binding.attn_kvcache_append_norm_rope(q, k, v, cache, other, slots, **how(c)), cache, other]
    for i, (groups, Hq, Hkv, d, ps, padding) in enumerate(SHARED):
        c = dev(shared_case(groups, Hq, Hkv, d, ps, seed=60 + i, padding=padding))
        out, lse = (torch.zeros(s, dtype=t, device="cuda") for s, t in (
            (c.q.shape, torch.bfloat16),
            ((c.q.shape[0], Hq) if c.cu_seqlens_q is None else (Hq, c.q.shape[0]), torch.float32)))
        got += call(binding, c, out=out, lse=lse)
    torch.cuda.synchronize()
    assert binding.attn_get_device_status() == 0
    return [t.cpu() for t in got]


def test_checked_build_gives_the_regular_results(request):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    attn_build.build()
    binding.load()
    regular = run()
    request.getfixturevalue("checked")
    for i, (a, b) in enumerate(zip(regular, run())):
        assert torch.equal(a, b), i
