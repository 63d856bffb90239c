"""fa_qk_norm_rope and its gradients against the formulas in 64 bits."""
import math

import pytest
import torch

from tests import decoder_testlib as lib

pytestmark = pytest.mark.gpu
EPS = 1e-6
F32 = 2.0 ** -24


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_attention_forward_02_gb300 as fa
    fa.fa_clear_status()
    yield fa
    assert fa.fa_last_status() == 0


def inputs(B, N, Hq, Hk, d, dtype, layout, seed=0, std=1.0):
    """q and k as slices of a fused projection, token-major or head-major tensors."""
    g = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()

    if layout == "fused":
        rows = normal(B, N, (Hq + 2 * Hk) * d)
        q, k = rows[..., :Hq * d].unflatten(-1, (Hq, d)), rows[..., Hq * d:(Hq + Hk) * d].unflatten(-1, (Hk, d))
    elif layout == "heads":
        q, k = normal(B, Hq, N, d).transpose(1, 2), normal(B, Hk, N, d).transpose(1, 2)
    else:
        q, k = normal(B, N, Hq, d), normal(B, N, Hk, d)
    w = [(1 + 0.2 * torch.randn(d, generator=g)).to(dtype).cuda() for _ in range(2)]
    return q, k, w[0], w[1], g


def rotation(B, N, rot, g):
    """A table, random rows of it for every token, and those rows."""
    if not rot:
        return None, None, None
    table = lib.rope_table(N + 77, rot).cuda()
    pos = torch.randint(0, N + 77, (B, N), generator=g, dtype=torch.int32).cuda()
    return table, pos, table[pos.long()][:, :, None]


def close(got, want, size, dtype):
    """One rounding of the output: u |y| (and a subnormal half step). In 32 bits before it: the sum of
    d <= 128 squares (relative error <= 8 levels of adds and 8 products, 17 units), the mean, the
    root (2 units and half the sum's error), the products with r and w (3), the rotation's two
    products and sum (3) of elements of magnitude up to `size`: under 24 units F32 of 2 size."""
    tol = lib.step(dtype) * want.abs() + lib.tiny(dtype) + 24 * F32 * (1 + lib.step(dtype)) * 2 * size
    err = (got.double() - want).abs()
    assert (err <= tol).all(), (err - tol).max()


CASES = [  # B, N, Hq, Hk, d, rot, interleaved, dtype, layout
    (1, 1, 1, 1, 64, 64, False, "bf16", "tokens"),
    (1, 1, 32, 8, 128, 128, False, "bf16", "fused"),
    (2, 7, 3, 1, 64, 16, True, "fp16", "heads"),
    (1, 33, 5, 5, 128, 64, True, "bf16", "fused"),
    (3, 333, 12, 12, 64, 32, False, "fp16", "fused"),
    (2, 100, 7, 2, 128, 16, False, "fp16", "heads"),
    (1, 64, 32, 8, 128, 0, False, "bf16", "fused"),
    (4, 1025, 8, 4, 64, 48, False, "bf16", "tokens"),
    (1, 4097, 16, 2, 128, 112, True, "fp16", "fused"),
    (1, 5000, 40, 8, 64, 64, True, "bf16", "heads"),
    (2, 3001, 2, 1, 64, 64, False, "fp16", "fused"),
    (3, 2047, 1, 1, 128, 32, True, "bf16", "heads"),
]


@pytest.mark.parametrize("B,N,Hq,Hk,d,rot,inter,dtype,layout", CASES)
def test_forward(fa, B, N, Hq, Hk, d, rot, inter, dtype, layout):
    q, k, wq, wk, g = inputs(B, N, Hq, Hk, d, lib.DTYPES[dtype], layout)
    table, pos, rows = rotation(B, N, rot, g)
    qo, ko = fa.qk_norm_rope(q, k, wq, wk, table, pos, EPS, inter)
    for x, w, y in ((q, wq, qo), (k, wk, ko)):
        want, size = lib.norm_rope64(x, w, rows, EPS, inter)
        close(y, want, size, x.dtype)


def test_default_positions_in_place_and_head_major_outputs(fa):
    q, k, wq, wk, _ = inputs(2, 40, 6, 2, 128, torch.bfloat16, "fused")
    table = lib.rope_table(40, 128).cuda()
    rows = table[None, :, None]
    want = [lib.norm_rope64(x, w, rows, EPS, False) for x, w in ((q, wq), (k, wk))]
    out = [torch.full((2, H, 40, 128), math.nan, dtype=q.dtype, device="cuda") for H in (6, 2)]
    qo, ko = fa.qk_norm_rope(q, k, wq, wk, table, q_out=out[0].transpose(1, 2), k_out=out[1].transpose(1, 2))
    close(qo, *want[0], q.dtype)
    close(ko, *want[1], q.dtype)
    fa.qk_norm_rope(q, k, wq, wk, table, q_out=q, k_out=k)  # in place, inside the fused projection
    assert torch.equal(q, qo) and torch.equal(k, ko)


def test_small_and_large_values(fa):
    """Rows of zeros (eps alone under the root) and of the type's far ends."""
    q, k, wq, wk, _ = inputs(1, 9, 2, 2, 64, torch.bfloat16, "tokens")
    q[0, 0], q[0, 1], q[0, 2] = 0, 1e-20, 1e15
    k[0, 3:5] = 1e-4
    qo, ko = fa.qk_norm_rope(q, k, wq, wk, lib.rope_table(9, 64).cuda())
    rows = lib.rope_table(9, 64).cuda()[None, :, None]
    for x, w, y in ((q, wq, qo), (k, wk, ko)):
        close(y, *lib.norm_rope64(x, w, rows, EPS, False), x.dtype)


@pytest.mark.parametrize("B,N,Hq,Hk,d,rot,inter,dtype,layout", CASES)
def test_backward(fa, B, N, Hq, Hk, d, rot, inter, dtype, layout):
    dt = lib.DTYPES[dtype]
    q, k, wq, wk, g = inputs(B, N, Hq, Hk, d, dt, layout)
    dq_out, dk_out = inputs(B, N, Hq, Hk, d, dt, "tokens" if layout == "fused" else "heads", seed=9)[:2]
    table, pos, rows = rotation(B, N, rot, g)
    dq, dk, dwq, dwk = fa.qk_norm_rope_backward(dq_out, dk_out, q, k, wq, wk, table, pos, EPS, inter)
    again = fa.qk_norm_rope_backward(dq_out, dk_out, q, k, wq, wk, table, pos, EPS, inter)
    assert all(torch.equal(a, b) for a, b in zip((dq, dk, dwq, dwk), again))
    for go, x, w, dx, dw in ((dq_out, q, wq, dq, dwq), (dk_out, k, wk, dk, dwk)):
        want, wdw, mag, r = lib.norm_rope_grad64(go, x, w, rows, EPS, inter)
        # |dx| <= r (|u| + |x r| |mean|): 32-bit errors are a few tens of units of those magnitudes
        u = go.double().abs().amax(-1, keepdim=True) * 2 * w.double().abs().max()
        size = r * (u + (x.double() * r).abs().amax(-1, keepdim=True) * u)
        tol = lib.step(dt) * want.abs() + lib.tiny(dt) + 64 * F32 * size
        err = (dx.double() - want).abs()
        assert (err <= tol).all(), (err - tol).max()
        # a sum over rows in 32 bits: a chain of at most tokens*heads/(lanes) adds in registers, then a
        # tree; each term is off by under 32 units of its own magnitude
        chain = 32 + 64 + B * N * (Hq + Hk) / 128
        slack = mag + 2 * (go.double().abs().amax() * (x.double() * r).abs().amax())
        assert ((dw.double() - wdw).abs() <= chain * F32 * slack).all()


def test_backward_against_differences(fa):
    """(f(x + h v) - f(x - h v)) / 2h of f = <g, y> in 64 bits, along random directions."""
    q, k, wq, wk, g = inputs(1, 3, 2, 1, 64, torch.float16, "tokens")
    table, pos, rows = rotation(1, 3, 32, g)
    dq_out, dk_out = inputs(1, 3, 2, 1, 64, torch.float16, "tokens", seed=3)[:2]
    dq, dk, dwq, dwk = fa.qk_norm_rope_backward(dq_out, dk_out, q, k, wq, wk, table, pos, EPS, True)
    for go, x, w, dx, dw in ((dq_out, q, wq, dq, dwq), (dk_out, k, wk, dk, dwk)):
        f = lambda x, w: (lib.norm_rope64(x, w, rows, EPS, True)[0] * go.double()).sum()  # noqa: E731
        x, w, h = x.double(), w.double(), 1e-5
        for _ in range(3):
            v, z = torch.randn_like(x), torch.randn_like(w)
            slope = (f(x + h * v, w + h * z) - f(x - h * v, w - h * z)) / (2 * h)
            got = (dx.double() * v).sum() + (dw.double() * z).sum()
            # dx is rounded: at most u |dx| |v| a place; the difference's own error is O(h^2)
            tol = (lib.step(torch.float16) * dx.double().abs() * v.abs()).sum() + 1e-4
            assert (got - slope).abs() <= tol


def test_one_set_alone_and_no_rows(fa):
    q, k, wq, wk, _ = inputs(1, 5, 2, 2, 64, torch.float16, "tokens")
    none = k[:, :, :0]
    qo, ko = fa.qk_norm_rope(q, none, wq, wk)
    assert torch.equal(qo, fa.qk_norm_rope(q, k, wq, wk)[0]) and ko.shape == none.shape
    assert torch.equal(fa.qk_norm_rope(none, k, wq, wk)[1], fa.qk_norm_rope(q, k, wq, wk)[1])
    dq, dk, dwq, dwk = fa.qk_norm_rope_backward(none, k, none, k, wq, wk)
    assert not dwq.any() and dwk.abs().sum() > 0
    empty = q[:, :0]
    dq, dk, dwq, dwk = fa.qk_norm_rope_backward(empty, empty, empty, empty, wq, wk)
    assert dq.shape == empty.shape and not dwq.any() and not dwk.any()


def test_a_position_outside_the_table_is_reported_and_left_alone(fa):
    q, k, wq, wk, _ = inputs(1, 4, 2, 1, 64, torch.bfloat16, "tokens")
    table = lib.rope_table(6, 64).cuda()
    pos = torch.tensor([[0, 6, -1, 5]], dtype=torch.int32).cuda()
    out = [torch.full_like(x, 7.0) for x in (q, k)]
    fa.qk_norm_rope(q, k, wq, wk, table, pos, q_out=out[0], k_out=out[1])
    assert fa.fa_last_status() == fa.FA_ERR_RANGE
    fa.fa_clear_status()
    assert (out[0][:, 1:3] == 7).all() and (out[1][:, 1:3] == 7).all()
    good = torch.tensor([[0, 5]], dtype=torch.int32).cuda()
    want = fa.qk_norm_rope(q[:, ::3], k[:, ::3], wq, wk, table, good)
    assert torch.equal(out[0][:, ::3], want[0]) and torch.equal(out[1][:, ::3], want[1])
    grads = fa.qk_norm_rope_backward(q, k, q, k, wq, wk, table, pos, dq=out[0], dk=out[1])
    assert fa.fa_last_status() == fa.FA_ERR_RANGE
    fa.fa_clear_status()
    assert (out[0][:, 1:3] == 7).all()
    few = fa.qk_norm_rope_backward(q[:, ::3], k[:, ::3], q[:, ::3], k[:, ::3], wq, wk, table, good)
    assert torch.allclose(grads[2], few[2], rtol=1e-5, atol=1e-5)


def test_another_stream_and_a_captured_graph(fa):
    q, k, wq, wk, _ = inputs(2, 300, 4, 2, 128, torch.bfloat16, "fused")
    table = lib.rope_table(300, 128).cuda()
    want = fa.qk_norm_rope(q, k, wq, wk, table)
    grads = fa.qk_norm_rope_backward(*want, q, k, wq, wk, table)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fa.qk_norm_rope(q, k, wq, wk, table, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = fa.qk_norm_rope(q, k, wq, wk, table)
        back = fa.qk_norm_rope_backward(*y, q, k, wq, wk, table)
    for x in (*y, *back):
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*y, *back), (*want, *grads)))
