"""The range-checked build of the key weights and the eviction over 16-bit caches, and of all operators of a compact cache on
arrays that are not as they should be: no check of the kernels' own places fires (the status says what was passed over),
and results are the release build's bit by bit."""
import pytest
import torch

from tests import compact_testlib as c8
from tests import decoder_testlib as lib
from tests.test_compact_debug_gpu import FORMS, cache, done, libs, rows, stream  # noqa: F401

pytestmark = pytest.mark.gpu


def weigh_and_evict(fa, library, b, q, L, scales):
    B, T, kv = len(b.new), q.shape[0], cache(fa, b)
    ids = (b.cu_seqlens.data_ptr(), b.seq_lens.data_ptr(), b.block_table.data_ptr(), b.block_table.shape[1])
    w = torch.full((b.k_pages.shape[0], b.Hkv, b.page), 0.25, device="cuda")
    ks, vs = scales
    said = [done(fa, library, library.fa_paged_key_weights(
        kv, ks, rows(fa, q), L.data_ptr(), w.data_ptr(), B, T, b.max_q, *ids, b.d ** -0.5, 1, fa.FA_BF16, stream()))]
    budget = max(1, max(b.total) // 2)
    kept = torch.empty(B, b.Hkv, budget, dtype=torch.int32, device="cuda")
    now = torch.empty(B, dtype=torch.int32, device="cuda")
    n = library.fa_paged_evict_workspace_bytes(B, b.Hkv, budget, int(ks is not None))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    said.append(done(fa, library, library.fa_paged_evict(
        kv, ks, vs, w.data_ptr(), B, *ids[1:], budget, budget // 3, kept.data_ptr(), now.data_ptr(), ws.data_ptr(), n,
        stream())))
    return said, (b.k_pages.view(torch.uint8), b.v_pages.view(torch.uint8), w.view(torch.int32), kept, now)  # (bits: NaN is NaN)


@pytest.mark.parametrize("new,total,Hq,Hkv,d,page,wide", FORMS)
def test_weights_and_eviction_over_16_bits(libs, new, total, Hq, Hkv, d, page, wide):  # noqa: F811
    fa, rel, dbg = libs
    held = []
    for library in (rel, dbg):
        b = lib.Batch(new, total, Hkv, d, page, torch.bfloat16, seed=1, wide=wide, lead=1, behind=2)
        q = b.rows(Hq)
        L = lib.attend64(b, q, d ** -0.5, True)[1].float()
        said, got = weigh_and_evict(fa, library, b, q, L, (None, None))
        assert said == [0, 0], [fa.strerror(s) for s in said]
        held.append(got)
    assert all(torch.equal(x, y) for x, y in zip(*held))


@pytest.mark.parametrize("change", ["offsets", "pages", "lengths"])
def test_bad_arrays(libs, change):  # noqa: F811
    fa, rel, dbg = libs
    held = []
    for library in (rel, dbg):
        b = c8.Batch8([5, 1, 40, 2], [900, 60, 300, 41], 2, 64, 16, torch.bfloat16, seed=2, lead=1, behind=2)
        q, k, v = b.rows(8), b.rows(2), b.rows(2)
        L = c8.attend64(b, q, 0.125, True)[1].float()
        if change == "offsets":
            b.cu_seqlens[:] = torch.tensor([1, 40, 46, 3, 9], dtype=torch.int32)
        elif change == "pages":
            b.block_table[0, 3], b.block_table[2, 1], b.block_table[2, 18] = -1, 10 ** 6, b.k_pages.shape[0]
        else:
            b.seq_lens[:] = torch.tensor([2, 1 << 30, -9, 41], dtype=torch.int32)
        ids = (b.cu_seqlens.data_ptr(), b.seq_lens.data_ptr(), b.block_table.data_ptr(), b.block_table.shape[1])
        said = done(fa, library, library.fa_paged_append_fp8(
            cache(fa, b), b.k_scale.data_ptr(), b.v_scale.data_ptr(), rows(fa, k), rows(fa, v), 4, b.T, *ids, None, fa.FA_BF16,
            stream()))
        more, got = weigh_and_evict(fa, library, b, q, L, (b.k_scale.data_ptr(), b.v_scale.data_ptr()))
        assert said == fa.FA_ERR_RANGE and fa.FA_ERR_RANGE in more and fa.FA_ERR_BOUNDS not in more
        held.append((*got, b.k_scale, b.v_scale))
    assert all(torch.equal(x, y) for x, y in zip(*held))
