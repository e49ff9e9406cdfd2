"""The mixture-of-experts operators at the ends of their ranges, against formulas in 64 bits.

Tolerances count roundings as in test_experts_gpu.py: half a step of the output type relative to
the value (bf16 2^-8, e4m3 2^-4), 2^-14 for the fast exponential of SiLU and its slope.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from jagged_hstu_attention_02_b200 import ops

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# ------------------------------------------------------------------ SiLU far from zero

# rows of each expert, and the contraction, of the products' three kernels: single blocks (128 x 128
# tiles), pairs of blocks, blocks that share a tile's contraction.  16384 rows of two experts make
# pairs; 17 slices of the contraction and 12 tiles make 8 blocks share each.
KERNELS = {"single": ([100, 97], 1), "pair": ([11000, 9001], 1), "shared": ([64, 65], 17)}
WIDE = 512


def _far(lo, hi, n=WIDE):
    """[n] bf16 values: far ones of lo .. hi beside ordinary ones in neighbouring columns, on
    either side, and beside one another."""
    far = [lo, hi] + [float(v) for v in np.geomspace(abs(lo), abs(hi), 11)[1:-1] * np.sign(lo)]
    g = torch.Generator().manual_seed(11)
    v = torch.randn(n, generator=g) * 4
    f = torch.tensor(far)
    i = torch.arange(n)
    v = torch.where(i % 4 == 0, f[i // 4 % len(far)], v)              # far, ordinary
    v = torch.where(i % 8 == 7, f[(i // 8 + 5) % len(far)], v)        # ordinary, far
    v = torch.where(i % 16 == 1, f[(i // 16 + 3) % len(far)], v)      # far, far
    return v.to(BF)


def _silu64(v):
    v = v.double()
    return torch.where(v < -700, 0.0 * v, v / (1 + torch.exp(-v)))


def _slope64(v):
    """sigma(v) (1 + v (1 - sigma(v))); 1 and 0 far from zero, where the terms leave their range."""
    v = v.double()
    c = v.clamp(-700, 700)
    p = 1 / (1 + torch.exp(-c))
    return p * (1 + c / (1 + torch.exp(c)))


def _offsets(counts):
    return torch.tensor([0] + counts, device="cuda").cumsum(0)


def _far_product(kernel, v, e4m3):
    """Rows whose product with either expert's matrix is v in every row: (x, w, offsets), in 8 bits
    (x, its scales, w, its scales, offsets).  One term of the contraction is not zero, so the
    product is exact."""
    counts, slices = KERNELS[kernel]
    K = (16 if e4m3 else 8) if slices == 1 else slices * (128 if e4m3 else 64)
    S, E = sum(counts), len(counts)
    at = K - 3
    if e4m3:
        x = torch.zeros(S, K, device="cuda")
        w = torch.zeros(E, WIDE, K, device="cuda")
        x[:, at], w[:, :, at] = 2.0, 0.5
        ws = v.float().cuda().expand(E, WIDE).contiguous()
        return x.to(ops.F8), torch.ones(S, device="cuda"), w.to(ops.F8), ws, _offsets(counts)
    x, w = torch.zeros(S, K, device="cuda", dtype=BF), torch.zeros(E, K, WIDE, device="cuda", dtype=BF)
    x[:, at], w[:, at, :] = 1.0, v.cuda()
    return x, w, _offsets(counts)


def _rows_match(got, want, tol, what):
    got = got.double()
    bad = ~((got - want.cuda()).abs() <= tol.cuda())               # (NaN is bad)
    at = torch.nonzero(bad)
    assert not len(at), "%s: %g for %g at %s" % (
        what, got[tuple(at[0])], want[at[0][1]], tuple(at[0].tolist()))


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("lo,hi", [(-30.0, -60.0), (-100.0, -1e6), (-1e12, -3e38)])
def test_silu_and_its_slope_of_large_negative_values_go_to_zero(kernel, lo, hi):
    """Far down the result is 0, off by at most 43 2^-62 < 1e-17 where that begins."""
    v = _far(lo, hi)
    want = _silu64(v)
    tol = want.abs() * (2 ** -8 + 2 ** -14) + 1e-17
    x, w, off = _far_product(kernel, v, False)
    pre = torch.empty(x.shape[0], WIDE, dtype=BF, device="cuda")
    out = ops.expert_proj(x, w, off, silu=True, pre=pre)
    assert torch.equal(pre, v.cuda().expand_as(pre))
    _rows_match(out, want, tol, "silu")
    x, xs, w, ws, off = _far_product(kernel, v, True)
    _rows_match(ops.expert_proj_e4m3(x, xs, w, ws, off, silu=True), want, tol, "silu, 8 bits")
    _check_slope(kernel, v)


def _check_slope(kernel, v):
    counts, slices = KERNELS[kernel]
    N, S, E = 8 if slices == 1 else slices * 64, sum(counts), len(counts)
    dout, w = torch.zeros(S, N, device="cuda", dtype=BF), torch.zeros(E, WIDE, N, device="cuda", dtype=BF)
    dout[:, N - 3], w[:, :, N - 3] = 1.0, 1.5
    silu_pre = v.cuda().expand(S, WIDE).contiguous()
    dx, _ = ops.expert_proj_bwd(dout, torch.zeros_like(silu_pre), w, _offsets(counts), silu_pre=silu_pre,
                                grads=(torch.empty_like(silu_pre), None))
    # the slope is a sum of terms of at most 1.1, each within 2^-14 of its value
    want = 1.5 * _slope64(v)
    _rows_match(dx, want, want.abs() * 2 ** -8 + 1.5 * 2 ** -14 * (v.double().abs() < 43) *
                _slope_terms(v) + 1e-17, "slope")


def _slope_terms(v):
    c = v.double().clamp(-700, 700)
    p = 1 / (1 + torch.exp(-c))
    return p * (1 + c.abs() / (1 + torch.exp(c)))


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("lo,hi", [(20.0, 300.0), (1e3, 1e6), (1e7, 3e38)])
def test_silu_of_large_positive_values_is_the_value_and_its_slope_one(kernel, lo, hi):
    """Whatever stands in the column beside them."""
    v = _far(lo, hi)
    want = _silu64(v)
    x, w, off = _far_product(kernel, v, False)
    _rows_match(ops.expert_proj(x, w, off, silu=True), want, want.abs() * (2 ** -8 + 2 ** -14), "silu")
    _check_slope(kernel, v)


@pytest.mark.parametrize("kernel", KERNELS)
def test_silu_beside_values_that_are_not_finite(kernel):
    """NaN and infinities stay in their own columns; NaN stays NaN, and infinity itself."""
    v = _far(1.0, 5.0).float()
    i = torch.arange(WIDE)
    v[i % 8 == 2], v[i % 8 == 5], v[i % 8 == 7] = float("nan"), float("inf"), float("-inf")
    v = v.to(BF)
    plain = torch.isfinite(v.float())
    want = _silu64(torch.where(plain, v, torch.zeros_like(v)))
    x, w, off = _far_product(kernel, v, False)
    x8, xs, w8, ws, off = _far_product(kernel, v, True)
    for out in (ops.expert_proj(x, w, off, silu=True), ops.expert_proj_e4m3(x8, xs, w8, ws, off, silu=True)):
        _rows_match(out[:, plain], want[plain], want[plain].abs() * (2 ** -8 + 2 ** -14) + 1e-17, "silu")
        assert torch.isnan(out[:, v.isnan()]).all() and (out[:, v == float("inf")] == float("inf")).all()
    counts, slices = KERNELS[kernel]
    N, S, E = 8 if slices == 1 else slices * 64, sum(counts), len(counts)
    dout, w = torch.zeros(S, N, device="cuda", dtype=BF), torch.zeros(E, WIDE, N, device="cuda", dtype=BF)
    dout[:, N - 3], w[:, :, N - 3] = 1.0, 1.5
    pre = v.cuda().expand(S, WIDE).contiguous()
    dx = ops.expert_proj_bwd(dout, torch.zeros_like(pre), w, off, silu_pre=pre,
                             grads=(torch.empty_like(pre), None))[0]
    slope = 1.5 * _slope64(torch.where(plain, v, torch.zeros_like(v)))[plain]
    _rows_match(dx[:, plain], slope, slope.abs() * 2 ** -8 + 1.5 * 1.1 * 2 ** -14, "slope")
    assert torch.isnan(dx[:, v.isnan()]).all()


# ------------------------------------------------------------------ norm

def test_norm_without_residual_into_an_earlier_result_keeps_the_rows_themselves():
    """The sum of a norm without a residual is x: not what an earlier call left in `out`."""
    g = torch.Generator().manual_seed(3)
    x1, x2, res = ((torch.randn(40, 256, generator=g)).to(BF).cuda() for _ in range(3))
    w = (1 + 0.2 * torch.randn(256, generator=g)).cuda()
    dy = torch.randn(40, 256, generator=g).to(BF).cuda()
    for first in (ops.rms_norm_rows(x1, w, training=True), ops.rms_norm_rows(x1, w, res, training=True)):
        kept = x1.clone(), first.sum.clone()
        r = ops.rms_norm_rows(x2, w, training=True, out=first)
        fresh = ops.rms_norm_rows(x2, w, training=True)
        assert r.y is first.y and r.rstd is first.rstd             # written again
        assert torch.equal(r.y, fresh.y) and torch.equal(r.rstd, fresh.rstd)
        assert torch.equal(r.sum, x2)
        for a, b in zip(ops.rms_norm_rows_bwd(dy, r.sum, r.rstd, w),
                        ops.rms_norm_rows_bwd(dy, fresh.sum, fresh.rstd, w)):
            assert torch.equal(a, b)
        assert torch.equal(x1, kept[0]) and torch.equal(first.sum, kept[1])
    r = ops.rms_norm_rows(x2, w, res, training=True, out=ops.rms_norm_rows(x1, w, res, training=True))
    assert torch.equal(r.sum, ops.rms_norm_rows(x2, w, res).sum)


@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("rows,width", [(3, 512), (3, 509), (6000, 512), (6000, 509)])
def test_norm_e4m3_of_the_largest_and_smallest_values(rows, width, group):
    """y = weight here (rows of +-1, eps 0).  Groups with a maximum in (2^126, 2^128), where a
    fast division of 448 by it would give 0, and groups below 2^-100, whose scale is that of
    2^-100: 2^-100 / 448 within 2^-17."""
    g = torch.Generator().manual_seed(width)
    sign = (2 * torch.randint(0, 2, (rows, width), generator=g) - 1).float()
    for top in (3.4e38, 1.8e38, 9e37, 8e37, 1e-20, 1e-33):
        w = torch.rand(width, generator=g) * 0.9 * top
        w[::16] = top
        r = ops.rms_norm_rows(sign.cuda(), w.cuda(), eps=0.0, e4m3=True, group=group)
        y = (sign * w).double()
        want = torch.full((rows, r.scales.shape[1]), max(float(w.max()), 2.0 ** -100) / 448, dtype=torch.float64)
        assert ((r.scales.double().cpu() - want).abs() <= want * 2 ** -17).all(), top
        v = y / want[0, 0]
        got = r.y.float().double().cpu()
        tol = torch.maximum(v.abs() * 2 ** -4, torch.tensor(2.0 ** -10)) + v.abs() * 2 ** -17
        assert ((got - v).abs() <= tol).all(), (top, got[0, :4], v[0, :4])


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("rows,width", [(5183, 512), (9471, 464), (5980, 64), (9000, 1024), (9000, 2048), (5183, 499)])
def test_norm_weight_gradients_of_many_rows_every_time(rows, width, dtype):
    """More rows than groups of warps, several groups in a block: the blocks' parts meet in the memory
    of the rings.  The same call 100 times, each within its tolerance and with the same bits."""
    g = torch.Generator().manual_seed(rows)
    dy, h, dsum = (torch.randn(rows, width, generator=g).to(dtype).cuda() for _ in range(3))
    rstd = (h.double().pow(2).mean(1) + 1e-5).rsqrt().float()
    w = (1 + 0.2 * torch.randn(width, generator=g)).cuda()
    terms = dy.double() * h.double() * rstd.double()[:, None]
    want, tol = terms.sum(0), (rows + 64) * 2 ** -24 * terms.abs().sum(0)
    first = None
    for i in range(100):
        for d in (dsum, None):
            dw = ops.rms_norm_rows_bwd(dy, h, rstd, w, dsum=d)[1]
            assert ((dw.double() - want).abs() <= tol).all(), i
            first = dw if first is None else first
            assert torch.equal(dw, first), i


# ------------------------------------------------------------------ sort

_SORT = """
import numpy as np, torch
from jagged_hstu_attention_02_b200 import ops
rng = np.random.default_rng(1)
for n in (2000, 5000):
    for dtype in (np.int32, np.int64):
        for E in (639, 640, 700, 767, 768, 769, 1024):
            ids = rng.integers(-1, E, (n // 2, 2)).astype(dtype)
            r = ops.expert_sort(torch.from_numpy(ids).cuda(), E)
            flat = ids.reshape(-1)
            order = np.argsort(np.where(flat < 0, E, flat), kind="stable")
            m = int((flat >= 0).sum())
            slots = np.full(n, -1)
            slots[order[:m]] = np.arange(m)
            ends = np.concatenate([[0], np.cumsum(np.bincount(flat[flat >= 0], minlength=E))])
            assert np.array_equal(r.slots.cpu().numpy().reshape(-1), slots), (n, dtype, E)
            assert np.array_equal(r.offsets.cpu().numpy(), ends), (n, dtype, E)
            assert np.array_equal(r.rows.cpu().numpy()[:m], order[:m] // 2), (n, dtype, E)
print("sorted")
"""


def test_sort_of_any_number_of_experts_in_a_new_process():
    """The numbers of experts ascend: no earlier call has asked for more shared memory."""
    r = subprocess.run([sys.executable, "-c", _SORT], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "sorted" in r.stdout, r.stderr[-2000:]


# ------------------------------------------------------------------ dispatch

def test_dispatch_of_rows_without_elements_moves_their_scales():
    slots = torch.tensor([[2, 0], [-1, 1], [3, 9]], dtype=torch.int32, device="cuda")
    x = torch.empty(3, 0, dtype=BF, device="cuda")
    scales = torch.arange(12, device="cuda").float().view(3, 4)
    out, got = ops.expert_dispatch(x, slots, scales=scales, scales_out=torch.full((6, 4), -1.0, device="cuda"))
    want = torch.full((6, 4), -1.0, device="cuda")
    want[[2, 0, 1, 3]] = scales[[0, 0, 1, 2]]
    assert out.shape == (6, 0) and torch.equal(got, want)


# ------------------------------------------------------------------ combine

@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("width", [8, 64, 100, 520, 1001, 4096])
def test_combine_gradients_of_pairs_without_a_row_are_zero_whatever_dout_holds(width, dtype):
    """Padding tokens' rows of dout hold NaN and infinities; neither they nor other tokens' pairs
    without a row see them."""
    g = torch.Generator().manual_seed(width)
    T, k = 37, 3
    slots = torch.randperm(T * k, generator=g).int().view(T, k)
    slots[::4] = -1                                            # padding tokens
    slots[1::4, 1] = -1
    slots[2::4, 2] = T * k                                     # behind the rows
    y = torch.randn(T * k, width, generator=g).to(dtype)
    dout = torch.randn(T, width, generator=g).to(dtype)
    dout[::8], dout[4::8] = float("nan"), float("inf")
    w = torch.rand(T, k, generator=g)
    dy, dw = ops.expert_combine_bwd(dout.cuda(), y.cuda(), slots.cuda(), w.cuda(),
                                    grads=(torch.full_like(y, 7.0).cuda(), torch.full((T, k), 7.0).cuda()))
    dw = dw.double().cpu()
    live = (slots >= 0) & (slots < T * k)
    assert (dw[~live] == 0).all()
    rows = y.double()[slots.long().clamp(0, T * k - 1)]
    terms = dout.double()[:, None, :] * rows
    # a term's chain: the elements that a lane or thread adds, 5 shuffles and 8 warps
    tol = terms.abs().sum(2) * (width / 32 + 14) * 2 ** -24
    assert ((dw - terms.sum(2)).abs() <= tol)[live].all()
    named = torch.zeros(T * k, dtype=torch.bool)
    named[slots[live].long()] = True
    assert torch.isfinite(dy.float()).all() and (dy.cpu()[~named] == 7).all()


# ------------------------------------------------------------------ waits

@pytest.mark.parametrize("what", ["product", "gradients"])
@pytest.mark.parametrize("counts,K,N", [([9000, 1100], 512, 2056), ([64, 65], 4104, 136),
                                        ([64, 65], 136, 4104), ([5000], 64, 128), ([300, 200], 512, 256)],
                         ids=["pair", "shared", "shared gradient", "parts of the rows", "single"])
def test_a_wait_that_runs_out_is_reported_by_every_kernel(counts, K, N, what):
    """A planted wait that nothing satisfies runs out after a millisecond: the products on pairs of
    blocks, with a shared contraction and from parts of the rows say so and leave the GPU usable;
    the next call is right again."""
    g = torch.Generator().manual_seed(K)
    S, E = sum(counts), len(counts)
    x, do = (torch.randn(S, n, generator=g).to(BF).cuda() for n in (K, N))
    w = (torch.randn(E, K, N, generator=g) * K ** -0.5).to(BF).cuda()
    off = _offsets(counts)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call():
        if what == "product":
            return [ops.expert_proj(x, w, off, silu=True, status=status)]
        return ops.expert_proj_bwd(do, x, w, off, status=status)

    ref = call()
    torch.cuda.synchronize()
    assert status.item() == 0
    ops.set_wait_test(2_000_000, True)
    try:
        call()
        torch.cuda.synchronize()
    finally:
        ops.set_wait_test(0, False)
    assert status.item() == ops.DEV_WAIT_TIMEOUT
    status.zero_()
    for a, b in zip(call(), ref):
        assert torch.equal(a, b)
    assert status.item() == 0


# ------------------------------------------------------------------ the layer

@pytest.mark.parametrize("T,k,E,d,ff", [(300, 2, 8, 128, 256), (77, 3, 5, 144, 136), (1, 1, 1, 64, 64)])
def test_layer_in_8_bits_against_its_own_quantised_rows(T, k, E, d, ff):
    """What follows the norm's 8-bit rows, from those rows and their scales in 64 bits.  Two tensors on
    the way are rounded to bf16 and the output once more; a random product carries a relative
    error on with a factor of at most 2, so the layer's part of the output is within 4 2^-8 of its
    2-norm, and the output's rounding."""
    g = torch.Generator().manual_seed(T)

    def randn(*shape):
        return torch.randn(*shape, generator=g)

    x, res = randn(T, d).to(BF).cuda(), (2 * randn(T, d)).to(BF).cuda()
    nw = (1 + 0.1 * randn(d)).cuda()
    ids = torch.randint(0, E, (T, k), generator=g).int().cuda()
    gates = torch.softmax(randn(T, k), 1).cuda()
    wt = randn(E, ff, d) * d ** -0.5
    ws = wt.abs().amax(2) / 448
    wq, ws = (wt / ws[..., None]).to(ops.F8).cuda(), ws.cuda()
    w_out = (randn(E, ff, d) * ff ** -0.5).to(BF).cuda()
    s = ops.expert_layer_fwd(x, res, nw, ids, gates, (wq, ws), w_out)
    n = ops.rms_norm_rows(x, nw, res, e4m3=True)
    rows = n.y.double() * n.scales.double()
    part = torch.zeros(T, d, dtype=torch.float64, device="cuda")
    for j in range(k):
        for e in range(E):
            t = torch.nonzero(ids[:, j] == e).squeeze(1)
            pre = rows[t] @ (wq[e].double() * ws[e].double()[:, None]).T
            part[t] += gates[t, j, None].double() * ((pre * torch.sigmoid(pre)) @ w_out[e].double())
    got = s["o"].double() - s["sum"].double()
    assert torch.equal(s["sum"], n.sum)
    assert (got - part).norm() <= part.norm() * 4 * 2 ** -8 + s["o"].double().norm() * 2 ** -8
