"""The range-checked build (libfa_debug.so) of the operators of a compact cache: no check fires on shapes of every
kernel form, results are the release build's bit by bit, and a workspace cut through the test hook makes the checks
fire while nothing is written that they guard. The cut lies inside a real allocation of full size."""
import ctypes

import pytest
import torch

from tests import compact_testlib as c8

pytestmark = pytest.mark.gpu
FORMS = [  # new, total, Hq, Hkv, d, page, table width: single tokens, drafts, 17 to 128 rows, pairs of tiles
    ([1], [1001], 32, 8, 128, 16, None),
    ([1, 1, 1, 1], [3000, 20, 400, 2100], 8, 2, 64, 16, None),
    ([4, 2, 4], [5000, 700, 4], 8, 2, 128, 64, None),
    ([7, 9, 1], [5000, 700, 3], 6, 1, 128, 64, None),
    ([30, 1], [5000, 4000], 4, 4, 64, 16, None),
    ([60, 1, 20], [200, 2000, 60], 4, 2, 128, 16, 200),
    ([300, 40], [300, 500], 4, 2, 64, 64, None),
    ([257, 100, 5], [3000, 100, 300], 6, 2, 64, 16, None),
]


@pytest.fixture(scope="module")
def libs():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_attention_forward_02_gb300 as fa
    rel, dbg = fa.load_library(fa.LIB_PATH), fa.load_library(fa.DEBUG_LIB_PATH)
    assert dbg.fa_clear_status() == 0 and rel.fa_clear_status() == 0
    assert dbg.fa_debug_cap_workspace(-1) == 1
    yield fa, rel, dbg
    dbg.fa_debug_cap_workspace(-1)


def stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def cache(fa, b):
    s = b.k_pages.stride()
    return fa.fa_paged_kv(b.k_pages.data_ptr(), b.v_pages.data_ptr(), s[0], s[1], s[2], b.k_pages.shape[0], b.page, b.Hkv,
                          b.k_pages.shape[3])


def rows(fa, x):
    return fa.fa_heads(x.data_ptr(), 0, x.stride(0), x.stride(1), x.shape[1])


def done(fa, library, rc):
    assert rc == 0, fa.strerror(rc)
    torch.cuda.synchronize()
    status = library.fa_last_status()
    assert library.fa_clear_status() == 0
    return status


def attend(fa, library, b, q, causal, fill=99.0):
    """O, L, the workspace behind its records as bytes, and the status."""
    T, Hq, d = q.shape
    O, L = torch.full_like(q, fill), torch.full((T, Hq), fill, device="cuda")
    n = library.fa_fwd_paged_workspace_bytes(Hq, b.Hkv, d, b.max_q)
    ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
    status = done(fa, library, library.fa_fwd_paged_fp8(
        cache(fa, b), b.k_scale.data_ptr(), b.v_scale.data_ptr(), rows(fa, q), rows(fa, O), L.data_ptr(), len(b.new), T,
        b.max_q, b.cu_seqlens.data_ptr(), b.seq_lens.data_ptr(), b.block_table.data_ptr(), b.block_table.shape[1],
        d ** -0.5, int(causal), fa.FA_BF16, ws.data_ptr(), n, stream()))
    records = -(-torch.cuda.get_device_properties(0).multi_processor_count * 32 // 256) * 256
    return O, L, ws[records:], status


def batch(new, total, Hq, Hkv, d, page, wide):
    b = c8.Batch8(new, total, Hkv, d, page, torch.bfloat16, seed=1, wide=wide, lead=1, behind=2)
    return b, b.rows(Hq)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,total,Hq,Hkv,d,page,wide", FORMS)
def test_no_check_fires_and_results_match_release(libs, new, total, Hq, Hkv, d, page, wide, causal):
    fa, rel, dbg = libs
    b, q = batch(new, total, Hq, Hkv, d, page, wide)
    want, got = attend(fa, rel, b, q, causal), attend(fa, dbg, b, q, causal)
    assert want[3] == 0 and got[3] == 0, (fa.strerror(want[3]), fa.strerror(got[3]))
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("new,total,Hq,Hkv,d,page,wide", FORMS)
def test_a_cut_workspace_is_not_written_and_the_rest_is_right(libs, new, total, Hq, Hkv, d, page, wide):
    fa, rel, dbg = libs
    b, q = batch(new, total, Hq, Hkv, d, page, wide)
    want = attend(fa, rel, b, q, True)
    split = bool((want[2] != 0xA5).any())
    try:
        assert dbg.fa_debug_cap_workspace(0) == 1 and rel.fa_debug_cap_workspace(0) == 0
        cut, release = attend(fa, dbg, b, q, True), attend(fa, rel, b, q, True)
    finally:
        dbg.fa_debug_cap_workspace(-1)
    assert release[3] == 0 and torch.equal(release[0], want[0])  # the release build ignores the hook
    assert cut[3] == (fa.FA_ERR_BOUNDS if split else 0), fa.strerror(cut[3])
    assert (cut[2] == 0xA5).all()
    right, left = (cut[0] == want[0]).all(-1) & (cut[1] == want[1]), (cut[0] == 99).all(-1) & (cut[1] == 99)
    assert (right | left).all()
    again = attend(fa, dbg, b, q, True)
    assert again[3] == 0 and torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


@pytest.mark.parametrize("new,total,Hq,Hkv,d,page,wide", FORMS)
def test_append_weights_and_eviction_match_release(libs, new, total, Hq, Hkv, d, page, wide):
    fa, rel, dbg = libs
    held = []
    for library in (rel, dbg):
        b, q = batch(new, total, Hq, Hkv, d, page, wide)
        k, v = b.rows(Hkv), b.rows(Hkv)
        T, B, kv = q.shape[0], len(new), cache(fa, b)
        ids = (b.cu_seqlens.data_ptr(), b.seq_lens.data_ptr(), b.block_table.data_ptr(), b.block_table.shape[1])
        assert done(fa, library, library.fa_paged_append_fp8(
            kv, b.k_scale.data_ptr(), b.v_scale.data_ptr(), rows(fa, k), rows(fa, v), B, T, *ids, None, fa.FA_BF16,
            stream())) == 0
        _, L, _, _ = attend(fa, library, b, q, True)
        w = torch.full((b.k_pages.shape[0], Hkv, page), 0.25, device="cuda")
        assert done(fa, library, library.fa_paged_key_weights(
            kv, b.k_scale.data_ptr(), rows(fa, q), L.data_ptr(), w.data_ptr(), B, T, b.max_q, *ids, d ** -0.5, 1,
            fa.FA_BF16, stream())) == 0
        budget = max(1, max(total) // 2)
        kept = torch.empty(B, Hkv, budget, dtype=torch.int32, device="cuda")
        now = torch.empty(B, dtype=torch.int32, device="cuda")
        n = library.fa_paged_evict_workspace_bytes(B, Hkv, budget, 1)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        assert done(fa, library, library.fa_paged_evict(
            kv, b.k_scale.data_ptr(), b.v_scale.data_ptr(), w.data_ptr(), B, *ids[1:], budget, budget // 3,
            kept.data_ptr(), now.data_ptr(), ws.data_ptr(), n, stream())) == 0
        held.append((b.k_pages.view(torch.uint8), b.v_pages.view(torch.uint8), b.k_scale, b.v_scale, w, kept, now))
    assert all(torch.equal(x, y) for x, y in zip(*held))
