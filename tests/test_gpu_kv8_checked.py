"""The bounds-checking debug build on the 8-bit cache's calls: on valid inputs its extra checks stay
silent and its results are those of the regular build."""
import pytest
import torch

from tests.kv8_exact import kv8_case
from tests.test_gpu_checked_build import checked  # noqa: F401

pytestmark = pytest.mark.gpu


def test_checked_8bit_cache(checked):  # noqa: F811
    for q in ([3, 1], [200, 90]):  # the 16-row kernel, the staged path
        c = kv8_case([300, 40], q, 32, 8, 64, 32, seed=720, rotary_dim=64, spread=0.5)
        args = [t.cuda() for t in (c.q, c.k_new, c.v_new, *c.cache, c.cache_seqlens, c.block_table,
                                   c.cu_seqlens_q)]
        out, lse = checked.attn_fwd_kvcache_fp8(*args, max(q), 340 + sum(q), c.scale, True, -1, -1,
                                                c.rotary_cos.cuda(), c.rotary_sin.cuda())
        lens = torch.tensor([300 + q[0], 40 + q[1]], dtype=torch.int32).cuda()
        o1, l1 = checked.attn_decode_kvcache_fp8(args[0][:2], *args[3:7], lens, args[8])
        torch.cuda.synchronize()
        assert checked.attn_get_device_status() == 0
        for t in (out, lse, o1, l1):
            assert torch.isfinite(t.float()).all()
