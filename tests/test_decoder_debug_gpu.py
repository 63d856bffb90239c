"""The range-checked build (libfa_debug.so) of the paged attention: no check fires on shapes of every
kernel form, results are the release build's bit by bit, and a workspace cut through the test hook
makes the checks fire while nothing is written that they guard. The cut lies inside a real
allocation of full size."""
import ctypes

import pytest
import torch

from tests import decoder_testlib as lib

pytestmark = pytest.mark.gpu
FORMS = [  # new, total, Hq, Hkv, d, page, table width
    ([1], [1001], 32, 8, 128, 16, None),
    ([1, 1, 1, 1], [3000, 20, 400, 2100], 8, 2, 64, 16, None),
    ([7, 9, 1], [5000, 700, 3], 6, 1, 128, 64, None),
    ([60, 1, 20], [200, 2000, 60], 4, 2, 128, 16, 200),
    ([300, 40], [300, 500], 4, 2, 64, 64, None),
    ([300], [6000], 4, 1, 128, 64, None),
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


def run(fa, library, b, q, causal, fill=99.0):
    """O, L, the workspace behind its records as bytes, and the status."""
    T, Hq, d = q.shape
    O, L = torch.full_like(q, fill), torch.full((T, Hq), fill, device="cuda")
    n = library.fa_fwd_paged_workspace_bytes(Hq, b.Hkv, d, b.max_q)
    ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
    k = b.k_pages.stride()
    heads = [fa.fa_heads(x.data_ptr(), 0, x.stride(0), x.stride(1), Hq) for x in (q, O)]
    kv = fa.fa_paged_kv(b.k_pages.data_ptr(), b.v_pages.data_ptr(), k[0], k[1], k[2], b.k_pages.shape[0], b.page, b.Hkv, d)
    rc = library.fa_fwd_paged(kv, *heads, L.data_ptr(), len(b.new), T, b.max_q, b.cu_seqlens.data_ptr(),
                              b.seq_lens.data_ptr(), b.block_table.data_ptr(), b.block_table.shape[1], d ** -0.5,
                              int(causal), fa.FA_BF16 if q.dtype == torch.bfloat16 else fa.FA_F16, ws.data_ptr(), n,
                              ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0, fa.strerror(rc)
    torch.cuda.synchronize()
    records = -(-torch.cuda.get_device_properties(0).multi_processor_count * 32 // 256) * 256
    status = library.fa_last_status()
    assert library.fa_clear_status() == 0
    return O, L, ws[records:], status


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,total,Hq,Hkv,d,page,wide", FORMS)
def test_no_check_fires_and_results_match_release(libs, new, total, Hq, Hkv, d, page, wide, causal):
    fa, rel, dbg = libs
    b = lib.Batch(new, total, Hkv, d, page, torch.bfloat16, seed=1, wide=wide, lead=1, behind=2)
    q = b.rows(Hq)
    want, got = run(fa, rel, b, q, causal), run(fa, dbg, b, q, causal)
    assert want[3] == 0 and got[3] == 0, (fa.strerror(want[3]), fa.strerror(got[3]))
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("new,total,Hq,Hkv,d,page,wide", FORMS)
def test_a_cut_workspace_is_not_written_and_the_rest_is_right(libs, new, total, Hq, Hkv, d, page, wide):
    """No room for partial states: no byte of them is written, rows whose item lies in one range are
    right, the others are left as they were; without the cut the call is right again."""
    fa, rel, dbg = libs
    b = lib.Batch(new, total, Hkv, d, page, torch.bfloat16, seed=1, wide=wide, lead=1, behind=2)
    q = b.rows(Hq)
    want = run(fa, rel, b, q, True)
    split = bool((want[2] != 0xA5).any())
    try:
        assert dbg.fa_debug_cap_workspace(0) == 1 and rel.fa_debug_cap_workspace(0) == 0
        cut, release = run(fa, dbg, b, q, True), run(fa, rel, b, q, True)
    finally:
        dbg.fa_debug_cap_workspace(-1)
    assert release[3] == 0 and torch.equal(release[0], want[0])  # the release build ignores the hook
    assert cut[3] == (fa.FA_ERR_BOUNDS if split else 0), fa.strerror(cut[3])
    assert (cut[2] == 0xA5).all()
    right, left = (cut[0] == want[0]).all(-1) & (cut[1] == want[1]), (cut[0] == 99).all(-1) & (cut[1] == 99)
    assert (right | left).all()
    again = run(fa, dbg, b, q, True)
    assert again[3] == 0 and torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


def test_a_workspace_cut_in_the_middle(libs):
    """Pieces that fit are stored, none behind the cut; items with a piece behind it are left out."""
    fa, rel, dbg = libs
    b = lib.Batch([1, 1, 1, 1], [9000, 6000, 400, 7000], 2, 64, 16, torch.bfloat16, seed=4)
    q = b.rows(8)
    want = run(fa, rel, b, q, True)
    cap = want[2].numel() // 4 // 2
    try:
        assert dbg.fa_debug_cap_workspace(cap) == 1
        cut = run(fa, dbg, b, q, True)
    finally:
        dbg.fa_debug_cap_workspace(-1)
    assert cut[3] == fa.FA_ERR_BOUNDS and (cut[2][cap * 4:] == 0xA5).all() and (cut[2][:cap * 4] != 0xA5).any()
    right, left = (cut[0] == want[0]).all(-1) & (cut[1] == want[1]), (cut[0] == 99).all(-1) & (cut[1] == 99)
    assert (right | left).all() and right.any() and left.any()
