"""Scales of K and magnitudes of q near the ends of 32-bit numbers, in opposite directions, so that scores are ordinary ones:
attention and key weights over an 8-bit cache against 64 bits."""
import pytest
import torch

from tests import compact_testlib as c8
from tests.test_evict_gpu import check_weigh, fa  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,new", [(4, 2, 1), (8, 1, 2), (8, 2, 8), (4, 2, 60), (4, 2, 200)])
@pytest.mark.parametrize("power", [-100, -80, 80, 100])
def test_scores_are_what_counts(fa, power, Hq, Hkv, new):  # noqa: F811
    b = c8.Batch8([new, 0], [500, 70], Hkv, 64, 64, torch.bfloat16, seed=new, fill=0.0)
    q = (b.rows(Hq).double() * 2.0 ** power).bfloat16()
    used = b.k_scale > 2.0 ** -20  # (the others are pages of nobody)
    b.k_scale[used] = (b.k_scale[used].double() * 2.0 ** -power).float()
    assert torch.isfinite(q).all() and (b.k_scale > 0).all() and torch.isfinite(b.k_scale).all()
    b.decode()
    O, L = fa.attention_paged_fp8(q, b.k_pages, b.v_pages, b.k_scale, b.v_scale, b.block_table, b.cu_seqlens, b.seq_lens,
                                  b.max_q)
    want, lse, tol_o, tol_l = c8.attend64(b, q, 0.125, True)
    assert fa.fa_last_status() == 0
    assert ((O.double() - want).abs() <= tol_o).all() and ((L.double() - lse).abs() <= tol_l).all()
    check_weigh(fa, b, q, True)


@pytest.mark.parametrize("Hq,Hkv,new", [(4, 2, 1), (8, 2, 8), (4, 2, 200)])
@pytest.mark.parametrize("power", [-90, 90])
def test_values_near_the_ends(fa, power, Hq, Hkv, new):  # noqa: F811
    b = c8.Batch8([new, 0], [500, 70], Hkv, 64, 64, torch.bfloat16, seed=new, fill=0.0, odd=True)
    q = b.rows(Hq)
    b.v_scale.copy_((b.v_scale.double() * 2.0 ** power).clamp(min=2.0 ** -100).float())
    b.decode()
    O, L = fa.attention_paged_fp8(q, b.k_pages, b.v_pages, b.k_scale, b.v_scale, b.block_table, b.cu_seqlens, b.seq_lens,
                                  b.max_q)
    want, lse, tol_o, tol_l = c8.attend64(b, q, 0.125, True)
    assert fa.fa_last_status() == 0
    assert ((O.double() - want).abs() <= tol_o).all() and ((L.double() - lse).abs() <= tol_l).all()
