"""Refusals of the decoder-block operators: every check runs on the host before any CUDA call,
so fake pointers and CPU tensors do; and the plain 64-bit forms the GPU tests compare with are
themselves checked against autograd and against the attention oracle."""
import ctypes
import math

import pytest
import torch

import exact_attention_forward_02_gb300 as fa
from tests import decoder_testlib as lib

P = 1 << 20  # 16-byte aligned, not null, never touched


def heads(ptr=P, bs=0, ts=256, hs=64, H=4):
    return fa.fa_heads(ptr, bs, ts, hs, H)


def cache(k=P, v=P, ps=16384, hs=1024, ts=64, pages=8, page=16, Hkv=4, d=64):
    return fa.fa_paged_kv(k, v, ps, hs, ts, pages, page, Hkv, d)


def rope(table=P, length=64, rot=64):
    return fa.fa_rope(table, length, rot, 0)


def norm(q=None, k=None, qo=None, ko=None, B=1, N=8, d=64, wq=P, wk=P, eps=1e-6, rp=None, pos=None, dt=1):
    return fa.fa_qk_norm_rope(q or heads(), k or heads(), qo or heads(), ko or heads(), B, N, d, wq, wk, eps, rp,
                              pos, dt, None)


@pytest.mark.parametrize("args,code", [
    (dict(dt=2), "FA_ERR_DTYPE"),
    (dict(d=96), "FA_ERR_HEAD_DIM"),
    (dict(B=-1), "FA_ERR_SHAPE"),
    (dict(N=-1), "FA_ERR_SHAPE"),
    (dict(eps=-1.0), "FA_ERR_RANGE"),
    (dict(eps=math.nan), "FA_ERR_RANGE"),
    (dict(eps=math.inf), "FA_ERR_RANGE"),
    (dict(rp=rope(rot=24)), "FA_ERR_RANGE"),
    (dict(rp=rope(rot=128)), "FA_ERR_RANGE"),
    (dict(rp=rope(rot=-16)), "FA_ERR_RANGE"),
    (dict(rp=rope(length=-1)), "FA_ERR_RANGE"),
    (dict(rp=rope(table=P + 4)), "FA_ERR_ALIGN"),
    (dict(q=heads(ptr=None)), "FA_ERR_NULL"),
    (dict(ko=heads(ptr=None)), "FA_ERR_NULL"),
    (dict(q=heads(ptr=P + 8)), "FA_ERR_ALIGN"),
    (dict(k=heads(ts=260)), "FA_ERR_ALIGN"),
    (dict(qo=heads(hs=68)), "FA_ERR_ALIGN"),
    (dict(qo=heads(bs=4)), "FA_ERR_ALIGN"),
    (dict(qo=heads(H=5)), "FA_ERR_SHAPE"),
    (dict(q=heads(H=-1), qo=heads(H=-1)), "FA_ERR_SHAPE"),
    (dict(wq=None), "FA_ERR_NULL"),
    (dict(wk=P + 2), "FA_ERR_ALIGN"),
    (dict(pos=P + 2), "FA_ERR_ALIGN"),
    (dict(B=1 << 30, N=1 << 30), "FA_ERR_SHAPE"),
    (dict(N=0, wq=None, q=heads(ptr=None), qo=heads(ptr=None)), "FA_OK"),
    (dict(q=heads(None, H=0), k=heads(None, H=0), qo=heads(None, H=0), ko=heads(None, H=0), wq=None, wk=None),
     "FA_OK"),
])
def test_norm_rope_refusals(args, code):
    rc = norm(**args)
    assert rc == getattr(fa, code), fa.strerror(rc)


def norm_bwd(n=None, dwq=P, dwk=P, ws=P, nbytes=None, d=64, **sets):
    s = {name: sets.get(name) or heads() for name in ("dq_out", "dk_out", "q", "k", "dq", "dk")}
    return fa.fa_qk_norm_rope_bwd(s["dq_out"], s["dk_out"], s["q"], s["k"], s["dq"], s["dk"], dwq, dwk, 1, 8, d, P, P,
                                  1e-6, None, None, 1, ws,
                                  fa.fa_qk_norm_rope_bwd_workspace_bytes(d) if nbytes is None else nbytes, None)


@pytest.mark.parametrize("args,code", [
    (dict(dwq=None), "FA_ERR_NULL"),
    (dict(dwk=None), "FA_ERR_NULL"),
    (dict(dwk=P + 1), "FA_ERR_ALIGN"),
    (dict(ws=None), "FA_ERR_WORKSPACE"),
    (dict(nbytes=64), "FA_ERR_WORKSPACE"),
    (dict(ws=P + 4), "FA_ERR_ALIGN"),
    (dict(dq=heads(H=3)), "FA_ERR_SHAPE"),
    (dict(dk_out=heads(ptr=None)), "FA_ERR_NULL"),
    (dict(d=80, nbytes=1 << 20), "FA_ERR_HEAD_DIM"),
])
def test_norm_rope_bwd_refusals(args, code):
    rc = norm_bwd(**args)
    assert rc == getattr(fa, code), fa.strerror(rc)


def append(kv=None, k=None, v=None, B=2, T=8, cu=P, lens=P, table=P, width=4, rp=None, dt=1):
    return fa.fa_paged_append(kv or cache(), k or heads(), v or heads(), B, T, cu, lens, table, width, rp, dt, None)


CACHE_FAULTS = [
    (dict(kv=cache(d=96)), "FA_ERR_HEAD_DIM"),
    (dict(kv=cache(page=0)), "FA_ERR_RANGE"),
    (dict(kv=cache(page=4)), "FA_ERR_RANGE"),
    (dict(kv=cache(page=24)), "FA_ERR_RANGE"),
    (dict(kv=cache(page=192)), "FA_ERR_RANGE"),
    (dict(kv=cache(page=-16)), "FA_ERR_RANGE"),
    (dict(kv=cache(pages=-1)), "FA_ERR_SHAPE"),
    (dict(kv=cache(k=None)), "FA_ERR_NULL"),
    (dict(kv=cache(v=P + 8)), "FA_ERR_ALIGN"),
    (dict(kv=cache(ps=16388)), "FA_ERR_ALIGN"),
    (dict(kv=cache(hs=1028)), "FA_ERR_ALIGN"),
    (dict(kv=cache(ts=68)), "FA_ERR_ALIGN"),
    (dict(B=-1), "FA_ERR_SHAPE"),
    (dict(T=-1), "FA_ERR_SHAPE"),
    (dict(width=-1), "FA_ERR_SHAPE"),
    (dict(cu=None), "FA_ERR_NULL"),
    (dict(lens=None), "FA_ERR_NULL"),
    (dict(table=None), "FA_ERR_NULL"),
    (dict(cu=P + 2), "FA_ERR_ALIGN"),
    (dict(dt=5), "FA_ERR_DTYPE"),
    (dict(B=0, cu=None, lens=None, table=None), "FA_OK"),
    (dict(T=0, cu=None, lens=None, table=None), "FA_OK"),
]


@pytest.mark.parametrize("args,code", CACHE_FAULTS + [
    (dict(k=heads(H=3)), "FA_ERR_SHAPE"),
    (dict(v=heads(ptr=None)), "FA_ERR_NULL"),
    (dict(k=heads(hs=20)), "FA_ERR_ALIGN"),
    (dict(rp=rope(rot=72)), "FA_ERR_RANGE"),
])
def test_append_refusals(args, code):
    rc = append(**args)
    assert rc == getattr(fa, code), fa.strerror(rc)


def attend(kv=None, q=None, O=None, L=P, B=2, T=8, max_q=4, cu=P, lens=P, table=P, width=4, scale=0.125, causal=1,
           dt=1, ws=P, nbytes=1 << 40):
    return fa.fa_fwd_paged(kv or cache(), q or heads(H=8), O or heads(H=8), L, B, T, max_q, cu, lens, table, width,
                           scale, causal, dt, ws, nbytes, None)


@pytest.mark.parametrize("args,code", CACHE_FAULTS + [
    (dict(q=heads(H=8, ptr=P + 2)), "FA_ERR_ALIGN"),
    (dict(O=heads(H=8, ts=4)), "FA_ERR_ALIGN"),
    (dict(O=heads(H=8, ptr=None)), "FA_ERR_NULL"),
    (dict(O=heads(H=4)), "FA_ERR_SHAPE"),
    (dict(q=heads(H=6), O=heads(H=6)), "FA_ERR_SHAPE"),       # 4 key heads
    (dict(q=heads(H=1024), O=heads(H=1024)), "FA_ERR_SHAPE"),  # 256 query heads a key head
    (dict(kv=cache(Hkv=0)), "FA_ERR_SHAPE"),
    (dict(max_q=0), "FA_ERR_SHAPE"),
    (dict(kv=cache(pages=0)), "FA_ERR_SHAPE"),
    (dict(scale=-1.0), "FA_ERR_SCALE"),
    (dict(scale=math.nan), "FA_ERR_SCALE"),
    (dict(L=P + 2), "FA_ERR_ALIGN"),
    (dict(q=heads(H=0, ptr=None), O=heads(H=0, ptr=None)), "FA_OK"),
])
def test_attention_refusals(args, code):
    rc = attend(**args)
    assert rc == getattr(fa, code), fa.strerror(rc)


def _paged(dtype=torch.float16, device="cpu"):
    b = lib.Batch([2, 1], [20, 3], 2, 64, 16, dtype, device=device, fill=0.0)
    return b, b.rows(4, device=device)


def test_bindings_refuse_what_the_kernels_would_misread():
    b, q = _paged()
    table = (b.block_table, b.cu_seqlens, b.seq_lens)
    with pytest.raises(ValueError, match="CUDA"):
        fa.attention_paged(q, b.k_pages, b.v_pages, *table, 2)
    with pytest.raises(TypeError):
        fa.attention_paged(q.float(), b.k_pages, b.v_pages, *table, 2)
    with pytest.raises(TypeError):
        fa.attention_paged(q, b.k_pages, b.v_pages.bfloat16(), *table, 2)
    with pytest.raises(ValueError, match="strides"):
        fa.attention_paged(q, b.k_pages, b.v_pages.transpose(1, 2).contiguous().transpose(1, 2), *table, 2)
    with pytest.raises(TypeError, match="int32"):
        fa.attention_paged(q, b.k_pages, b.v_pages, b.block_table.long(), b.cu_seqlens, b.seq_lens, 2)
    with pytest.raises(ValueError, match="cu_seqlens"):
        fa.attention_paged(q, b.k_pages, b.v_pages, b.block_table, b.cu_seqlens[:2], b.seq_lens, 2)
    with pytest.raises(ValueError, match="block_table"):
        fa.attention_paged(q, b.k_pages, b.v_pages, b.block_table[:1], b.cu_seqlens, b.seq_lens, 2)
    with pytest.raises(ValueError, match="adjacent"):
        fa.attention_paged(q.transpose(0, 2).contiguous().transpose(0, 2), b.k_pages, b.v_pages, *table, 2)
    with pytest.raises(ValueError, match="out"):
        fa.attention_paged(q, b.k_pages, b.v_pages, *table, 2, out=q[:1])
    with pytest.raises(ValueError, match="overlap"):
        fa.attention_paged(q, b.k_pages, b.v_pages, *table, 2, out=q[:1].expand(3, 4, 64))
    with pytest.raises(ValueError, match="lse"):
        fa.attention_paged(q, b.k_pages, b.v_pages, *table, 2, lse=torch.zeros(4, 3))
    with pytest.raises(ValueError, match="workspace"):
        fa.attention_paged(q, b.k_pages, b.v_pages, *table, 2, workspace=torch.zeros(8))
    k = b.rows(2, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        fa.paged_append(k, k, b.k_pages, b.v_pages, *table)
    with pytest.raises(ValueError, match="heads"):
        fa.paged_append(q, q, b.k_pages, b.v_pages, *table)
    with pytest.raises(ValueError, match="v must be"):
        fa.paged_append(k, k[:1], b.k_pages, b.v_pages, *table)
    with pytest.raises(ValueError, match="rope"):
        fa.paged_append(k, k, b.k_pages, b.v_pages, *table, rope=torch.zeros(9, 40))
    x, w = torch.zeros(1, 5, 2, 64).half(), torch.zeros(64).half()
    with pytest.raises(ValueError, match="CUDA"):
        fa.qk_norm_rope(x, x, w, w)
    with pytest.raises(ValueError, match=r"\[B, N, H, d\]"):
        fa.qk_norm_rope(x, x[:, :4], w, w)
    with pytest.raises(TypeError):
        fa.qk_norm_rope(x, x, w.float(), w)
    with pytest.raises(ValueError, match="wq"):
        fa.qk_norm_rope(x, x, w[:32], w)
    with pytest.raises(TypeError, match="int32"):
        fa.qk_norm_rope(x, x, w, w, positions=torch.zeros(1, 5, dtype=torch.int64))
    with pytest.raises(ValueError, match="k_out"):
        fa.qk_norm_rope(x, x, w, w, k_out=x[:, :2])
    with pytest.raises(ValueError, match="dq_out"):
        fa.qk_norm_rope_backward(x[:, :2], x, x, x, w, w)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 16, 64])
def test_plain_gradients_are_autograd_s(rot, interleaved):
    torch.manual_seed(1)
    x = torch.randn(2, 3, 4, 64, dtype=torch.float64, requires_grad=True)
    w = torch.randn(64, dtype=torch.float64, requires_grad=True)
    g = torch.randn(2, 3, 4, 64, dtype=torch.float64)
    rows = lib.rope_table(9, rot)[torch.tensor([[0, 3, 8], [1, 1, 2]])][:, :, None] if rot else None
    y, _ = lib.norm_rope64(x, w, rows, 1e-6, interleaved)
    y.backward(g)
    dx, dw, _, _ = lib.norm_rope_grad64(g, x.detach(), w.detach(), rows, 1e-6, interleaved)
    assert torch.allclose(dx, x.grad, rtol=1e-12, atol=1e-12)
    assert torch.allclose(dw, w.grad, rtol=1e-12, atol=1e-12)


def test_plain_attention_is_the_oracle_s(oracle_mod):
    """One sequence whose cache is all new: the dense causal attention of the oracle."""
    import numpy as np

    b = lib.Batch([9], [9], 2, 64, 16, torch.float16, device="cpu", fill=0.0)
    q = b.rows(4, device="cpu")
    for causal in (False, True):
        O, L, tol_o, _ = lib.attend64(b, q, 0.125, causal)
        k, v = (x[0].double().repeat_interleave(2, 0)[None].numpy() for x in (b.keys, b.values))
        Or, Lr = oracle_mod.attention(q.double().transpose(0, 1)[None].contiguous().numpy(), k, v, 0.125, causal)
        assert np.abs(O.transpose(0, 1).numpy() - Or[0]).max() < 1e-12
        assert np.abs(L.transpose(0, 1).numpy() - Lr[0]).max() < 1e-12
        assert (tol_o > 0).all()


def test_struct_layouts_match_the_header():
    """The ctypes structures have the C compiler's sizes and offsets on a 64-bit machine."""
    assert ctypes.sizeof(fa.fa_heads) == 40 and fa.fa_heads.H.offset == 32
    assert ctypes.sizeof(fa.fa_paged_kv) == 56 and fa.fa_paged_kv.num_pages.offset == 40
    assert ctypes.sizeof(fa.fa_rope) == 24 and fa.fa_rope.interleaved.offset == 16
