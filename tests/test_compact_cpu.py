"""Refusals of the operators of a compact cache: every check runs on the host before any CUDA call, so fake
pointers and CPU tensors do; and the plain 64-bit forms that the GPU tests compare with, checked by themselves."""
import math

import pytest
import torch

import exact_attention_forward_02_gb300 as fa
from tests import compact_testlib as c8
from tests import decoder_testlib as lib
from tests.test_decoder_cpu import cache, heads, rope

P = 1 << 20  # 16-byte aligned, not null, never touched


def ok(rc, code):
    assert rc == getattr(fa, code), fa.strerror(rc)


# a cache's own checks, in bytes where it holds 8 bits
CACHE = [
    (dict(kv=cache(d=96)), "FA_ERR_HEAD_DIM"),
    (dict(kv=cache(page=0)), "FA_ERR_RANGE"),
    (dict(kv=cache(page=24)), "FA_ERR_RANGE"),
    (dict(kv=cache(page=192)), "FA_ERR_RANGE"),
    (dict(kv=cache(pages=-1)), "FA_ERR_SHAPE"),
    (dict(kv=cache(k=None)), "FA_ERR_NULL"),
    (dict(kv=cache(k=P + 8)), "FA_ERR_ALIGN"),
    (dict(B=-1), "FA_ERR_SHAPE"),
    (dict(width=-1), "FA_ERR_SHAPE"),
    (dict(lens=None), "FA_ERR_NULL"),
    (dict(table=None), "FA_ERR_NULL"),
    (dict(lens=P + 2), "FA_ERR_ALIGN"),
    (dict(B=(1 << 30) + 1), "FA_ERR_SHAPE"),
    (dict(B=0, lens=None, table=None), "FA_OK"),
]
V = [(dict(kv=cache(v=None)), "FA_ERR_NULL"), (dict(kv=cache(v=P + 8)), "FA_ERR_ALIGN")]
STRIDES8 = [(dict(kv=cache(ps=16392)), "FA_ERR_ALIGN"), (dict(kv=cache(hs=1032)), "FA_ERR_ALIGN"),
            (dict(kv=cache(ts=72)), "FA_ERR_ALIGN")]  # multiples of 8, not of 16
ROWS = [(dict(cu=None), "FA_ERR_NULL"), (dict(cu=P + 1), "FA_ERR_ALIGN"), (dict(T=-1), "FA_ERR_SHAPE"),
        (dict(T=0, cu=None, lens=None, table=None), "FA_OK"), (dict(dt=5), "FA_ERR_DTYPE")]


def append(kv=None, ks=P, vs=P, k=None, v=None, B=2, T=8, cu=P, lens=P, table=P, width=4, rp=None, dt=1):
    return fa.fa_paged_append_fp8(kv or cache(), ks, vs, k or heads(), v or heads(), B, T, cu, lens, table, width, rp,
                                  dt, None)


@pytest.mark.parametrize("args,code", CACHE + V + STRIDES8 + ROWS + [
    (dict(ks=None), "FA_ERR_NULL"),
    (dict(vs=None), "FA_ERR_NULL"),
    (dict(vs=P + 2), "FA_ERR_ALIGN"),
    (dict(k=heads(H=3)), "FA_ERR_SHAPE"),
    (dict(v=heads(ptr=None)), "FA_ERR_NULL"),
    (dict(k=heads(hs=20)), "FA_ERR_ALIGN"),
    (dict(rp=rope(rot=72)), "FA_ERR_RANGE"),
    (dict(T=1 << 29), "FA_ERR_SHAPE"),  # 2^32 rows of k and v
])
def test_append_refusals(args, code):
    ok(append(**args), code)


def attend(kv=None, ks=P, vs=P, q=None, O=None, L=P, B=2, T=8, max_q=4, cu=P, lens=P, table=P, width=64, scale=0.125,
           causal=1, dt=1, ws=P, nbytes=1 << 40):
    return fa.fa_fwd_paged_fp8(kv or cache(), ks, vs, q or heads(H=8), O or heads(H=8), L, B, T, max_q, cu, lens, table,
                               width, scale, causal, dt, ws, nbytes, None)


QUERIES = [
    (dict(q=heads(H=8, ptr=P + 2)), "FA_ERR_ALIGN"),
    (dict(q=heads(H=8, ptr=None)), "FA_ERR_NULL"),
    (dict(kv=cache(Hkv=0)), "FA_ERR_SHAPE"),
    (dict(max_q=0), "FA_ERR_SHAPE"),
    (dict(kv=cache(pages=0)), "FA_ERR_SHAPE"),
    (dict(scale=-1.0), "FA_ERR_SCALE"),
    (dict(scale=math.nan), "FA_ERR_SCALE"),
    (dict(L=P + 2), "FA_ERR_ALIGN"),
    (dict(ks=P + 2), "FA_ERR_ALIGN"),
]


@pytest.mark.parametrize("args,code", CACHE + V + STRIDES8 + ROWS + QUERIES + [
    (dict(ks=None), "FA_ERR_NULL"),
    (dict(vs=None), "FA_ERR_NULL"),
    (dict(O=heads(H=4)), "FA_ERR_SHAPE"),
    (dict(q=heads(H=6), O=heads(H=6)), "FA_ERR_SHAPE"),        # 4 key heads
    (dict(q=heads(H=1024), O=heads(H=1024)), "FA_ERR_SHAPE"),  # 256 query heads a key head
    (dict(ws=P + 16), "FA_ERR_ALIGN"),
])
def test_attention_refusals(args, code):
    ok(attend(**args), code)


def weigh(kv=None, ks=P, q=None, L=P, w=P, B=2, T=8, max_q=4, cu=P, lens=P, table=P, width=4, scale=0.125, causal=1,
          dt=1):
    return fa.fa_paged_key_weights(kv or cache(), ks, q or heads(H=8), L, w, B, T, max_q, cu, lens, table, width, scale,
                                   causal, dt, None)


@pytest.mark.parametrize("args,code", CACHE + STRIDES8 + ROWS + QUERIES + [
    (dict(L=None), "FA_ERR_NULL"),
    (dict(w=None), "FA_ERR_NULL"),
    (dict(w=P + 2), "FA_ERR_ALIGN"),
    (dict(q=heads(H=6)), "FA_ERR_SHAPE"),
    (dict(q=heads(H=1024)), "FA_ERR_SHAPE"),
    (dict(ks=None, kv=cache(ts=68)), "FA_ERR_ALIGN"),
])
def test_key_weights_refusals(args, code):
    ok(weigh(**args), code)


def evict(kv=None, ks=P, vs=P, w=P, B=2, lens=P, table=P, width=4, budget=16, recent=4, kept=P, now=P, ws=P,
          nbytes=1 << 50):
    return fa.fa_paged_evict(kv or cache(), ks, vs, w, B, lens, table, width, budget, recent, kept, now, ws, nbytes, None)


@pytest.mark.parametrize("args,code", CACHE + V + STRIDES8 + [
    (dict(ks=None), "FA_ERR_NULL"),
    (dict(vs=None), "FA_ERR_NULL"),
    (dict(w=None), "FA_ERR_NULL"),
    (dict(kept=None), "FA_ERR_NULL"),
    (dict(now=None), "FA_ERR_NULL"),
    (dict(kept=P + 2), "FA_ERR_ALIGN"),
    (dict(w=P + 1), "FA_ERR_ALIGN"),
    (dict(budget=0), "FA_ERR_SHAPE"),
    (dict(recent=-1), "FA_ERR_SHAPE"),
    (dict(recent=17), "FA_ERR_SHAPE"),
    (dict(budget=0x7fffffff), "FA_ERR_SHAPE"),
    (dict(B=1 << 24), "FA_ERR_SHAPE"),  # 2^26 heads
    (dict(ws=None), "FA_ERR_WORKSPACE"),
    (dict(ws=P + 16), "FA_ERR_ALIGN"),
    (dict(nbytes=fa.fa_paged_evict_workspace_bytes(2, 4, 16, True) - 1), "FA_ERR_WORKSPACE"),
    (dict(kv=cache(Hkv=0)), "FA_OK"),
])
def test_evict_refusals(args, code):
    ok(evict(**args), code)


def test_workspace_sizes():
    size = fa.fa_paged_evict_workspace_bytes
    assert size(0, 4, 16, 1) == size(2, 0, 16, 1) == size(2, 4, 0, 1) == 0 == size(-1, 4, 16, 1)
    assert size(2, 4, 1000, 0) >= 2 * 4 * 1000 * 8 and size(2, 4, 1000, 1) >= size(2, 4, 1000, 0) + 2 * 4 * 1000 * 8
    assert size(300, 64, 1 << 20, 1) > 1 << 36  # 64-bit arithmetic


def _batch():
    b = c8.Batch8([2, 1], [20, 3], 2, 64, 16, torch.float16, device="cpu", fill=0.0)
    return b, b.rows(4, device="cpu"), (b.block_table, b.cu_seqlens, b.seq_lens)


def test_tensor_calls_of_the_8_bit_cache_refuse():
    b, q, table = _batch()
    cache8, k = (b.k_pages, b.v_pages, b.k_scale, b.v_scale), b.rows(2, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        fa.attention_paged_fp8(q, *cache8, *table, 2)
    with pytest.raises(TypeError, match="float8_e4m3fn"):
        fa.attention_paged_fp8(q, b.k_pages.half(), b.v_pages.half(), *cache8[2:], *table, 2)
    with pytest.raises(TypeError, match="float8_e4m3fn"):
        fa.attention_paged_fp8(q, b.k_pages.view(torch.float8_e5m2), *cache8[1:], *table, 2)
    with pytest.raises(TypeError):
        fa.attention_paged(q, *cache8[:2], *table, 2)  # the call for 16 bits
    with pytest.raises(TypeError, match="k_scale"):
        fa.attention_paged_fp8(q, *cache8[:2], b.k_scale.double(), b.v_scale, *table, 2)
    with pytest.raises(ValueError, match="v_scale"):
        fa.attention_paged_fp8(q, *cache8[:3], b.v_scale[:, :1], *table, 2)
    with pytest.raises(ValueError, match="v_scale"):
        fa.attention_paged_fp8(q, *cache8[:3], b.v_scale[:-1], *table, 2)
    with pytest.raises(TypeError, match="tensor"):
        fa.attention_paged_fp8(q, *cache8[:2], None, b.v_scale, *table, 2)
    with pytest.raises(ValueError, match="CUDA"):
        fa.paged_append_fp8(k, k, *cache8, *table)
    with pytest.raises(ValueError, match="heads"):
        fa.paged_append_fp8(q, q, *cache8, *table)
    with pytest.raises(TypeError):
        fa.paged_append_fp8(k.float(), k.float(), *cache8, *table)
    one = torch.zeros(1, 2, 16, 64, dtype=torch.uint8).expand(b.k_pages.shape[0], 2, 16, 64).view(torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="overlap"):
        fa.paged_append_fp8(k, k, one, one, *cache8[2:], *table)


def test_tensor_calls_of_key_weights_refuse():
    b, q, table = _batch()
    L, w = torch.zeros(q.shape[0], 4), torch.zeros(b.k_pages.shape[0], 2, 16)
    with pytest.raises(ValueError, match="CUDA"):
        fa.paged_key_weights(q, L, b.k_pages, w, *table, 2, k_scale=b.k_scale)
    with pytest.raises(TypeError):
        fa.paged_key_weights(q, L, b.k_pages, w, *table, 2)  # no scales: the cache must be q's type
    with pytest.raises(TypeError, match="float8_e4m3fn"):
        fa.paged_key_weights(q, L, b.k_pages.half(), w, *table, 2, k_scale=b.k_scale)
    with pytest.raises(TypeError, match="weights"):
        fa.paged_key_weights(q, L, b.k_pages, w.half(), *table, 2, k_scale=b.k_scale)
    with pytest.raises(ValueError, match="weights"):
        fa.paged_key_weights(q, L, b.k_pages, w[:, :, :8], *table, 2, k_scale=b.k_scale)
    with pytest.raises(ValueError, match="weights"):
        fa.paged_key_weights(q, L, b.k_pages, w.transpose(1, 2).contiguous().transpose(1, 2), *table, 2, k_scale=b.k_scale)
    with pytest.raises(ValueError, match="lse"):
        fa.paged_key_weights(q, L[:, :2], b.k_pages, w, *table, 2, k_scale=b.k_scale)


def test_tensor_calls_of_eviction_refuse():
    b, _, _ = _batch()
    w = torch.zeros(b.k_pages.shape[0], 2, 16)

    def call(budget=8, recent=2, kp=b.k_pages, vp=b.v_pages, ks=b.k_scale, vs=b.v_scale, **kw):
        fa.paged_evict(kp, vp, w, b.block_table, b.seq_lens, budget, recent, k_scale=ks, v_scale=vs, **kw)

    with pytest.raises(ValueError, match="CUDA"):
        call()
    with pytest.raises(ValueError, match="together"):
        call(vs=None)
    with pytest.raises(TypeError):
        call(ks=None, vs=None)  # an 8-bit cache without scales
    for budget, recent in ((0, 0), (8, 9), (8, -1), (-1, 0)):
        with pytest.raises(ValueError, match="budget"):
            call(budget, recent)
    with pytest.raises(ValueError, match="kept"):
        call(kept=torch.zeros(2, 2, 9, dtype=torch.int32))
    with pytest.raises(TypeError, match="kept"):
        call(kept=torch.zeros(2, 2, 8))
    with pytest.raises(ValueError, match="new_lens"):
        call(new_lens=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="workspace"):
        call(workspace=torch.zeros(8))
    with pytest.raises(ValueError, match="strides"):
        call(vp=b.v_pages.view(torch.uint8).transpose(1, 2).contiguous().transpose(1, 2).view(torch.float8_e4m3fn))


def test_plain_power_is_the_smallest_power_of_two_not_below():
    x = torch.tensor([1.0, 1.0 + 2 ** -30, 0.75, 2.0 ** -101, 0.0, 3e5 / 448], dtype=torch.float64)
    assert c8.power(x).tolist() == [1.0, 2.0, 1.0, c8.LEAST, c8.LEAST, 1024.0]


def test_plain_attention_over_codes_is_the_plain_one_over_their_values():
    """attend64 of an 8-bit batch against the 16-bit form over a cache that holds the same numbers."""
    b = c8.Batch8([3, 1, 0], [40, 5, 9], 2, 64, 16, torch.float32, device="cpu", seed=3)
    q = b.rows(4, device="cpu")
    want, got = lib.attend64(b, q, 0.2, True), c8.attend64(b, q, 0.2, True)
    assert torch.allclose(want[0], got[0], rtol=1e-12, atol=0) and torch.allclose(want[1], got[1], rtol=1e-12, atol=0)
