"""CPU checks of what the chunk call on the 8-bit cache makes of bounds far above the work itself: the
workspace follows the tokens of the call, not the bound."""
import pytest

from exact_attention_70_gb300 import binding
from exact_attention_70_gb300 import build as attn_build

MOST = 2 ** 31 - 1


@pytest.fixture(scope="module")
def need():
    attn_build.build()
    binding.load()

    def f(batch, total_q, max_q, total_k=4096, rotary=0, hq=32, hkv=8, d=128):
        return binding.attn_fwd_kvcache_fp8_workspace_bytes(batch, total_q, max_q, total_k, hq, hkv, d, 64, 64,
                                                            rotary)
    return f


@pytest.mark.parametrize("rotary", [0, 128])
@pytest.mark.parametrize("batch,total_q", [(1, 1), (8, 8), (64, 64), (8, 4096), (64, 600), (65535, 70000)])
def test_no_sequence_has_more_new_tokens_than_the_call(need, batch, total_q, rotary):
    want = need(batch, total_q, total_q, rotary=rotary)
    assert want > 0
    for bound in (total_q + 1, 10 ** 6, MOST):
        assert need(batch, total_q, bound, rotary=rotary) == want


def test_the_work_list_holds_the_tokens_of_the_call(need):
    """Tiles of 128 packed rows, at most one unfinished per sequence, 16 bytes an item and kv head."""
    batch, total_q, hkv, d = 65535, 70000, 8, 128
    staged_keys = (4096 + 128 * batch) * hkv * (2 * 2 * d + 2)        # f16 rows and scale bytes
    queries = total_q * 32 * (2 * 2 * d + 4)
    items = (total_q // 32 + batch) * hkv * 16
    assert need(batch, total_q, MOST, rotary=128) <= staged_keys + queries + items + batch * (2 * hkv + 4) * 4 + 8192


def test_workspace_grows_with_the_bound_until_the_tokens_are_reached(need):
    sizes = [need(64, 600, q) for q in (1, 64, 300, 600)]
    assert sizes == sorted(sizes)
