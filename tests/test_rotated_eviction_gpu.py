"""Rotated keys in a cache that is cut: queries and keys turned by the tokens' own positions (qk_norm_rope) and appended without
a table, against the definition in 64 bits over the kept tokens at the positions that they had."""
import math

import pytest
import torch

from tests import compact_testlib as c8
from tests import decoder_testlib as lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_attention_forward_02_gb300 as fa
    fa.fa_clear_status()
    return fa


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_tokens_after_an_eviction_stand_at_their_own_positions(fa, dtype, interleaved):
    Hq, Hkv, d, page, budget, recent, B = 8, 2, 64, 16, 150, 40, 2
    prompt = [400, 260]
    g = torch.Generator().manual_seed(5)
    make = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()  # noqa: E731
    rope = lib.rope_table(600, d).cuda()
    wq, wk = make(d).abs() + 0.5, make(d).abs() + 0.5
    wide = 30
    table = torch.randperm(B * wide + 2, generator=g)[:B * wide].int().view(B, wide).cuda()
    pages = B * wide + 2
    kp, vp = (torch.zeros(pages, Hkv, page, d, dtype=torch.uint8, device="cuda").view(c8.E4M3) for _ in range(2))
    ks, vs = (torch.ones(pages, Hkv, device="cuda") for _ in range(2))
    w = torch.zeros(pages, Hkv, page, device="cuda")
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    def step(q, k, v, positions, cu, lens, n):
        q, k = fa.qk_norm_rope(q[None], k[None], wq, wk, rope=rope, positions=positions[None], interleaved=interleaved)
        q, k = q[0], k[0]
        fa.paged_append_fp8(k, v, kp, vp, ks, vs, table, cu, lens)
        out, lse = fa.attention_paged_fp8(q, kp, vp, ks, vs, table, cu, lens, n)
        fa.paged_key_weights(q, lse, kp, w, table, cu, lens, n, k_scale=ks)
        return out

    T = sum(prompt)
    pos = torch.cat([torch.arange(n) for n in prompt]).int().cuda()
    lens, cu = ints(prompt), ints([0, prompt[0], T])
    k_raw, v_raw = make(T, Hkv, d), make(T, Hkv, d)
    step(make(T, Hq, d), k_raw, v_raw, pos, cu, lens, max(prompt))
    kept, lens = fa.paged_evict(kp, vp, w, table, lens, budget, recent, k_scale=ks, v_scale=vs)
    norm = lambda x, weight, at: lib.norm_rope64(x, weight, rope[at.long()][:, None], 1e-6, interleaved)[0]  # noqa: E731
    keys = [norm(k_raw[a:b], wk, pos[a:b]) for a, b in ((0, prompt[0]), (prompt[0], T))]
    keys = [torch.stack([keys[i][kept[i, h].long(), h] for h in range(Hkv)]) for i in range(B)]  # [Hkv, budget, d]
    cu = ints([0, 1, 2])
    for n in range(20):
        lens = lens + 1
        at = ints([prompt[0] + n, prompt[1] + n])
        q, k, v = make(B, Hq, d), make(B, Hkv, d), make(B, Hkv, d)
        out = step(q, k, v, at, cu, lens, 1)
        q64, k64 = norm(q, wq, at), norm(k, wk, at)
        t = budget + n + 1
        for i in range(B):
            keys[i] = torch.cat([keys[i], k64[i][:, None]], 1)
            used = table[i, :-(-t // page)].long()
            held = [(p.view(torch.uint8)[used].view(c8.E4M3).double() * s[used].double()[..., None, None]).transpose(0, 1)
                    .flatten(1, 2)[:, :t] for p, s in ((kp, ks), (vp, vs))]
            # the cache holds the keys at their own positions: one rounding of the 16-bit type, then two of E4M3 (the append's
            # and the move's under a scale that grew) and, of what is small, half a step of its subnormal numbers twice
            unit = ks[used].double().repeat_interleave(page, 0)[:t].T[..., None]
            off = keys[i].abs() * (2 * c8.HALF8 + 2.0 ** -6) + 2 * c8.TINY8 * unit
            assert ((held[0] - keys[i]).abs() <= off).all()
            # and the rows attend to what it holds: scores off by the rounding of the rotated q, weights by that much, one of O
            x = q64[i].view(Hkv, Hq // Hkv, d)
            s = x @ held[0].transpose(1, 2) / math.sqrt(d)
            p = s.softmax(-1)
            u = lib.step(dtype)
            e = 2 * u * (x.abs() @ held[0].abs().transpose(1, 2)).amax(-1, keepdim=True) / math.sqrt(d)
            want = p @ held[1]
            tol = (2 * e.exp().sub(1) + 2.0 ** -10) * (p @ held[1].abs()) + u * want.abs() + 2.0 ** -20
            assert ((out[i].double().view_as(want) - want).abs() <= tol).all()
    assert fa.fa_last_status() == 0
