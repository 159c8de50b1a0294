"""The step's calls together, as a serving loop and a training step use them."""
import pytest
import torch

from exact_attention_70_gb300 import synth
from oracle import oracle
from tests import step_exact
from tests.test_gpu_plan import attn  # noqa: F401

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def test_a_serving_loop(attn):  # noqa: F811
    """A prompt in the cache, three requests that go on from its pages with chunks and then single tokens,
    places, rows and attention from the step's calls alone; every step's attention over what was written,
    in 64 bits."""
    Hq, Hkv, d, ps, rot, prompt = 8, 2, 128, 16, 64, 160
    gen = torch.Generator().manual_seed(1)
    B, pages = 3, 64
    kc = torch.full((pages, ps, Hkv, d), float("nan"), dtype=BF16, device="cuda")
    vc = kc.clone()
    free = torch.randperm(pages, generator=gen).int().cuda()
    count = torch.tensor([pages], dtype=torch.int32, device="cuda")
    cos, sin = (t.cuda() for t in synth.rotary_tables(400, rot))
    weights = [(1 + 0.2 * torch.randn(d, generator=gen)).to(BF16).cuda() for _ in range(2)]
    keys, values = [None] * B, [None] * B  # what each sequence holds, as it was written

    def tokens(n):
        return (torch.randn((n, Hq + 2 * Hkv, d), generator=gen) * 2).to(BF16).cuda()

    def place(table, lens, new, total):
        cu, after, pos, slots, left = attn.attn_kvcache_plan(
            lens, torch.tensor(new, dtype=torch.int32, device="cuda"), table, free, count, ps, pages, total)
        count.copy_(left)
        x = tokens(total)
        q = attn.attn_kvcache_append_norm_rope(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], kc, vc, slots,
                                               *weights, rotary_cos=cos, rotary_sin=sin, positions=pos)
        k = attn.attn_qk_norm_rope(x[:, :Hq], x[:, Hq:Hq + Hkv], *weights, rotary_cos=cos, rotary_sin=sin,
                                   positions=pos)[1]
        return cu, after, q, k, x[:, Hq + Hkv:]

    # the prompt, as the only sequence; its pages lead the three requests' rows
    one = torch.full((1, 24), -1, dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    _, _, _, k, v = place(one, zero, [prompt], prompt)
    keys, values = [k] * B, [v] * B
    table = torch.full((B, 24), -1, dtype=torch.int32, device="cuda")
    table[:, :prompt // ps] = one[:, :prompt // ps]
    lens = torch.full((B,), prompt, dtype=torch.int32, device="cuda")
    group, prefix = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, B], [prompt]))
    for new, pad in (([5, 1, 40], 3), ([1, 1, 1], 0), ([1, 1, 1], 0), ([2, 0, 17], 0), ([1, 1, 1], 0)):
        total = sum(new) + pad
        cu, after, q, k, v = place(table, lens, new, total)
        single = new == [1, 1, 1]
        out, lse = attn.attn_decode_kvcache_shared(q, kc, vc, after, table, group, prefix,
                                                   None if single else cu, max(new))
        lens, at = after, 0
        for b, n in enumerate(new):
            keys[b], values[b] = torch.cat((keys[b], k[at:at + n])), torch.cat((values[b], v[at:at + n]))
            at += n
        assert lens.tolist() == [x.shape[0] for x in keys]
        c = step_exact.SharedCase(q.cpu(), kc.cpu(), vc.cpu(), lens.cpu(), table.cpu(), group.cpu(), prefix.cpu(),
                                  cu.cpu(), new, lens.tolist(), d ** -0.5, ps, max(new))
        ref = step_exact.shared_exact(c)
        n = sum(new)
        step_exact.shared_check(out[:n], (lse if single else lse.t())[:n], [r[:n] for r in ref])
        for b in range(B):  # the cache holds what was written, token by token
            j = torch.arange(keys[b].shape[0], device="cuda")
            page = table[b].long()[j // ps]
            assert torch.equal(kc[page, j % ps], keys[b]) and torch.equal(vc[page, j % ps], values[b])
        # the other calls on the same cache agree
        if single:
            o2, l2 = attn.attn_decode_kvcache(q, kc, vc, after, table)
            step_exact.shared_check(o2, l2, ref)
    assert attn.attn_get_device_status() == 0


def test_a_training_step(attn):  # noqa: F811
    """Norm and rotation, attention, both backward passes: the gradient of the projection's rows and of both
    weights along a random direction against differences of the whole in 64 bits.

    What the chain rounds to bf16 on the way (rotated rows, weights of attention, outputs, gradients: eight
    roundings of 2^-8 of values of either sign) moves the slope by a random walk over thousands of elements;
    2^-4 of the root of the sum of squares of the slope's terms is 16 roundings' worth, all of one sign."""
    T, Hq, Hkv, d, rot = 130, 4, 2, 64, 32
    gen = torch.Generator().manual_seed(2)
    x = torch.randn((T, Hq + 2 * Hkv, d), generator=gen).to(BF16)
    w = [1 + 0.2 * torch.randn(d, generator=gen) for _ in range(2)]
    g = torch.randn((T, Hq, d), generator=gen).to(BF16)
    cos, sin = synth.rotary_tables(64, rot)
    pos = torch.randint(0, 64, (3, T), generator=gen).int()
    sections = (4, 6, 6)
    turn = step_exact.turn_of(cos, sin, pos, 3, sections, False, False)
    cu = torch.tensor([0, 50, T], dtype=torch.int32)
    how = dict(q_weight=w[0].cuda(), k_weight=w[1].cuda(), rotary_cos=cos.cuda(), rotary_sin=sin.cuda(),
               positions=pos.cuda(), sections=sections)
    xg = x.cuda()
    q, k, v = xg[:, :Hq], xg[:, Hq:Hq + Hkv], xg[:, Hq + Hkv:].contiguous()
    qr, kr = attn.attn_qk_norm_rope(q, k, **how)
    out, lse = attn.attn_fwd(qr, kr, v, cu.cuda(), cu.cuda(), 80, 80, causal=True)
    dqr, dkr, dv = attn.attn_bwd(qr, kr, v, out, g.cuda(), lse, cu.cuda(), cu.cuda(), 80, 80, causal=True)
    dx = torch.empty_like(xg)
    dx[:, Hq + Hkv:] = dv
    _, _, dqw, dkw = attn.attn_qk_norm_rope_bwd(dqr, dkr, q, k, dq=dx[:, :Hq], dk=dx[:, Hq:Hq + Hkv], **how)
    assert attn.attn_get_device_status() == 0

    def f(x, wq, wk):
        q = step_exact.norm_rope(x[:, :Hq], wq, 1e-6, turn)[0]
        k = step_exact.norm_rope(x[:, Hq:Hq + Hkv], wk, 1e-6, turn)[0]
        o, _ = oracle.attn_fwd(q.numpy(), k.numpy(), x[:, Hq + Hkv:].numpy(), cu.numpy(), cu.numpy(), d ** -0.5, True,
                               -1, -1)
        return (torch.from_numpy(o) * g.double()).sum()

    for _ in range(4):
        args = x.double(), w[0].double(), w[1].double()
        v = [torch.randn(a.shape, generator=gen, dtype=torch.float64) for a in args]
        for i, grad in enumerate((dx, dqw, dkw)):
            h = 1e-5
            up, down = list(args), list(args)
            up[i], down[i] = args[i] + h * v[i], args[i] - h * v[i]
            slope = (f(*up) - f(*down)) / (2 * h)
            terms = grad.cpu().double() * v[i]
            assert abs(slope - terms.sum()) <= 2.0 ** -4 * terms.norm() * 4, (i, slope, terms.sum())
