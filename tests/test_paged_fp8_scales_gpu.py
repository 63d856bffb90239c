"""Attention over an 8-bit cache whose pages' v_scale lie far apart, against 64 bits with the stated range: 11 bits of P v_scale,
no finer than 2^-28 of the largest weight times the largest scale."""
import pytest
import torch

from tests import compact_testlib as c8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_attention_forward_02_gb300 as fa
    fa.fa_clear_status()
    return fa


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("Hq,Hkv,new", [(4, 2, 1), (8, 1, 2), (8, 2, 8), (4, 2, 60), (4, 2, 200)])
@pytest.mark.parametrize("far", [8, 16, 20, 24, 28, 40, 80])
def test_scales_far_apart(fa, far, Hq, Hkv, new, dtype):
    """The first page's v_scale is 2^far times the others', and no row gives it weight: beyond 2^16 (2^20 with many rows)
    the others lose bits, and count no longer in the end."""
    d, page = 64, 64
    b = c8.Batch8([new, 0], [500, 70], Hkv, d, page, dtype, seed=far, fill=0.0)
    q = b.rows(Hq)
    q[..., 0] = 24.0  # against the first page's keys: scores of -24 448 / 8 below the others'
    first = b.block_table[:, 0].long()
    b.k_scale[first] = 1.0
    codes = b.k_pages.view(torch.uint8)
    codes[first, :, :, 0] = 0xFE  # -448
    b.v_scale.fill_(2.0 ** -far)
    b.v_scale[first] = 1.0
    b.decode()
    O, L = fa.attention_paged_fp8(q, b.k_pages, b.v_pages, b.k_scale, b.v_scale, b.block_table, b.cu_seqlens, b.seq_lens,
                                  b.max_q)
    want, lse, tol_o, tol_l = c8.attend64(b, q, d ** -0.5, True)
    assert fa.fa_last_status() == 0
    assert ((O.double() - want).abs() <= tol_o).all() and ((L.double() - lse).abs() <= tol_l).all()
