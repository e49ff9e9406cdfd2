"""The mixture-of-experts operators on the GPU against their fp64 oracle.

Tolerances, element by element, from the arithmetic (u = 2^-24, one fp32 rounding; HALF = half a
step of the output type relative to the value: bf16 2^-8, fp32 2^-24, e4m3 2^-4):
 - a sum of n terms in fp32 is off by at most n u sum|terms|, whatever its order; n counts the
   longest chain of additions that a term goes through;
 - sums of squares have no cancellation: rstd is off by at most (chain + 4) u relative, the
   chain being 16 elements of a thread, 5 shuffles and 32 warps, so y before its rounding
   is within 64 u = 2^-18 of its value, and the fp32 sum h within u of its own;
 - an e4m3 value is rounded once from such a y over such a scale: half a step, 2^-4 of the value
   or 2^-10 where steps are constant (below 2^-6), plus 2^-17 of the value;
 - products of bf16 or e4m3 values are exact in fp32; the tensor cores add them 16 or 32 at a
   time with an fp32 accumulator, each step within 2^-22 of the magnitudes it adds:
   (d_in / 16 + 4) 2^-22 sum|x w| over the contraction;
 - SiLU and its slope are at most 1.1 steep, and their fast exponential is within 2^-14.
"""
import numpy as np
import pytest
import torch

from jagged_hstu_attention_02_b200 import ops
from oracle import experts as ox

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, F32 = torch.bfloat16, torch.float32
GUARD = 64


def _np(t):
    if t.dtype == ops.F8:
        t = t.float()
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def _rand(seed, *shape, dtype=BF, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


class Guarded:
    """A tensor between two bands of a marker value, to show that nothing outside is written."""

    def __init__(self, shape, dtype, fill=None):
        n = int(np.prod(shape))
        self.pad = max(GUARD, 16)
        mark = 72                                    # a value of every type
        pad = self.pad - n % self.pad + self.pad
        self.buf = torch.full((self.pad + n + pad,), mark, device="cuda").to(dtype)
        self.t = self.buf[self.pad:self.pad + n].view(*shape)
        self.n, self.mark = n, mark
        if fill is not None:
            self.t.fill_(fill)

    def check(self, what):
        b = self.buf.float()
        assert (b[:self.pad] == self.mark).all() and (b[self.pad + self.n:] == self.mark).all(), what


def _close(got, ref, tol, what):
    got = _np(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, what
    assert np.isfinite(got).all(), what + ": non-finite values"
    err = np.abs(got - ref) - tol
    assert (err <= 0).all(), "%s: %g over its tolerance at %s" % (
        what, err.max(), np.unravel_index(err.argmax(), err.shape))


# ------------------------------------------------------------------ norm

NORM_SHAPES = [(1, 1), (3, 7), (5, 8), (9, 33), (130, 100), (17, 256), (1, 512), (33, 520),
               (4, 1000), (7, 1024), (300, 1032), (3, 2049), (2, 4096), (3, 5000), (2, 16384),
               (2, 16383)]


def _norm_inputs(rows, width, dtype, seed, residual=True, weight=True):
    x = _rand(seed, rows, width, dtype=dtype)
    r = _rand(seed + 1, rows, width, dtype=dtype, scale=3.0) if residual else None
    w = (1 + 0.2 * _rand(seed + 2, width, dtype=F32)) if weight else None
    return x, r, w


def _opt(t):
    return None if t is None else _np(t)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("residual,weight", [(True, True), (False, False), (True, False)])
@pytest.mark.parametrize("shape", NORM_SHAPES)
def test_norm(shape, residual, weight, dtype):
    rows, width = shape
    x, r, w = _norm_inputs(rows, width, dtype, 10 + rows + width, residual, weight)
    y, s = Guarded(shape, dtype), Guarded(shape, dtype)
    rstd = Guarded((rows,), F32)
    out = ops.RmsNorm(y.t, None, s.t, rstd.t)
    ops.rms_norm_rows(x, w, r, eps=1e-5, training=True, out=out)
    ry, rh, rr = ox.rms_norm(_np(x), _opt(r), _opt(w), 1e-5)
    _close(y.t, ry, np.abs(ry) * (HALF[dtype] + 2 ** -18), "y")
    _close(rstd.t, rr, rr * 2 ** -18, "rstd")
    if residual:
        _close(s.t, rh, np.abs(rh) * (HALF[dtype] + U), "sum")
    for g in (y, s, rstd):
        g.check("norm writes outside its buffers")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("shape", NORM_SHAPES)
def test_norm_e4m3(shape, group, dtype):
    rows, width = shape
    x, r, w = _norm_inputs(rows, width, dtype, 40 + rows + width)
    x[rows - 1], r[rows - 1] = 0, 0                     # a row of zeros: scale 0, zeros
    groups = -(-width // (group or width))
    y, s, sc = Guarded(shape, ops.F8), Guarded(shape, dtype), Guarded((rows, groups), F32)
    ops.rms_norm_rows(x, w, r, e4m3=True, group=group, out=ops.RmsNorm(y.t, sc.t, s.t, None))
    ry, rh, _ = ox.rms_norm(_np(x), _np(r), _np(w), 1e-5)
    rs = ox.e4m3_scales(ry, group)
    _close(sc.t, rs, rs * 2 ** -17, "scales")
    wide = np.repeat(rs, group or width, axis=1)[:, :width]
    v = np.divide(ry, wide, out=np.zeros_like(ry), where=wide > 0)
    _close(y.t, v, np.maximum(np.abs(v) * 2 ** -4, 2 ** -10) + np.abs(v) * 2 ** -17, "q")
    assert not _np(y.t)[rows - 1].any() and not _np(sc.t)[rows - 1].any()
    _close(s.t, rh, np.abs(rh) * (HALF[dtype] + U), "sum")
    for g in (y, s, sc):
        g.check("norm writes outside its buffers")


def test_norm_of_no_rows_and_non_finite_rows():
    r = ops.rms_norm_rows(torch.empty(0, 64, dtype=BF, device="cuda"), e4m3=True, training=True)
    assert r.y.shape == (0, 64) and r.scales.shape == (0, 1) and r.rstd.shape == (0,)
    x = _rand(3, 3, 256, dtype=F32)
    x[0, 5], x[1, 7] = float("nan"), float("inf")
    y = ops.rms_norm_rows(x).y
    q = ops.rms_norm_rows(x, e4m3=True)
    assert torch.isnan(y[0]).all() and torch.isnan(q.y.float()[0]).all()
    assert torch.isnan(y[1, 7]) and (y[1, :7] == 0).all()     # 1 / sqrt(inf) = 0, inf * 0 = NaN
    assert torch.isfinite(y[2]).all() and torch.isfinite(q.y.float()[2]).all()


def test_norm_in_place():
    x, r, w = _norm_inputs(37, 520, BF, 77)
    ref = ops.rms_norm_rows(x, w, r)
    stream = r.clone()
    y = torch.empty_like(x)
    ops.rms_norm_rows(x, w, stream, out=ops.RmsNorm(y, None, stream, None))
    assert torch.equal(y, ref.y) and torch.equal(stream, ref.sum)


def _norm_bwd_case(shape, dtype, seed, weight=True, dsum=True):
    rows, width = shape
    dy, h = _rand(seed, rows, width, dtype=dtype), _rand(seed + 1, rows, width, dtype=dtype)
    d = _rand(seed + 2, rows, width, dtype=dtype) if dsum else None
    w = (1 + 0.2 * _rand(seed + 3, width, dtype=F32)) if weight else None
    rstd = (1 / torch.sqrt((h.double() ** 2).mean(1) + 1e-5)).float()
    return dy, h, rstd, w, d


def _check_norm_bwd(dx, dw, dy, h, rstd, w, d, dtype):
    rows, width = dy.shape
    rdx, rdw = ox.rms_norm_bwd(_np(dy), _np(h), _np(rstd), _opt(w), _opt(d))
    xh = _np(h) * _np(rstd)[:, None]
    g = np.abs(_np(dy) * (1 if w is None else _np(w)))
    size = _np(rstd)[:, None] * (g + np.abs(xh) * (g * np.abs(xh)).mean(1, keepdims=True))
    size = size + (0 if d is None else np.abs(_np(d)))
    _close(dx, rdx, np.abs(rdx) * HALF[dtype] + size * 2 ** -18, "dx")
    if dw is not None:
        # a term's chain: its block's rows, up to 8 rows in parallel, 37 blocks, 8 strands
        chain = rows + 64
        _close(dw, rdw, chain * U * (np.abs(_np(dy)) * np.abs(xh)).sum(0), "dweight")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", NORM_SHAPES + [(3000, 64), (1111, 2056)])
def test_norm_bwd(shape, dtype):
    dy, h, rstd, w, d = _norm_bwd_case(shape, dtype, 5 + sum(shape))
    gx, gw = Guarded(shape, dtype), Guarded((shape[1],), F32)
    ops.rms_norm_rows_bwd(dy, h, rstd, w, dsum=d, grads=(gx.t, gw.t))
    _check_norm_bwd(gx.t, gw.t, dy, h, rstd, w, d, dtype)
    gx.check("dx")
    gw.check("dweight")
    again = ops.rms_norm_rows_bwd(dy, h, rstd, w, dsum=d)
    assert torch.equal(again[0], gx.t) and torch.equal(again[1], gw.t)      # deterministic


def test_norm_bwd_parts_left_out_and_in_place():
    for weight, dsum in ((False, True), (True, False), (False, False)):
        dy, h, rstd, w, d = _norm_bwd_case((70, 640), BF, 9, weight, dsum)
        dx, dw = ops.rms_norm_rows_bwd(dy, h, rstd, w, dsum=d)
        assert (dw is None) == (not weight)
        _check_norm_bwd(dx, dw, dy, h, rstd, w, d, BF)
    dy, h, rstd, w, d = _norm_bwd_case((70, 640), BF, 9)
    ref = ops.rms_norm_rows_bwd(dy, h, rstd, w, dsum=d)
    for into in (dy.clone(), d.clone()):
        a = (into, d) if torch.equal(into, dy) else (dy, into)
        dx, _ = ops.rms_norm_rows_bwd(a[0], h, rstd, w, dsum=a[1],
                                      grads=(into, torch.empty_like(w)))
        assert torch.equal(dx, ref[0])
    # a weight gradient without rows is zero
    e = torch.empty(0, 640, dtype=BF, device="cuda")
    _, dw = ops.rms_norm_rows_bwd(e, e, torch.empty(0, device="cuda"), w)
    assert not dw.any()


# more rows than groups of warps, rows that start anywhere: they arrive through the ring
MANY_ROWS = [(20001, 1), (9001, 7), (5003, 33), (5000, 499), (2999, 1001), (1501, 2001), (700, 4085),
             (333, 8001), (301, 16383)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", MANY_ROWS)
def test_norm_of_many_rows_that_start_anywhere(shape, dtype):
    test_norm(shape, True, True, dtype)
    test_norm(shape, False, False, dtype)
    test_norm_e4m3(shape, 0, dtype)
    test_norm_e4m3(shape, 32, dtype)
    test_norm_bwd(shape, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", [(9001, 7), (5003, 33), (2999, 1001), (301, 16383)])
def test_norm_rows_do_not_see_their_neighbours(shape, dtype):
    x, r, w = _norm_inputs(*shape, dtype, 5)
    clean = ops.rms_norm_rows(x, w, r, training=True)
    q = ops.rms_norm_rows(x, w, r, e4m3=True, group=64)
    dirty = x.clone()
    dirty[::2] = float("nan")
    d = ops.rms_norm_rows(dirty, w, r, training=True)
    dq = ops.rms_norm_rows(dirty, w, r, e4m3=True, group=64)
    for a, b in ((clean.y, d.y), (clean.sum, d.sum), (clean.rstd, d.rstd), (q.y, dq.y), (q.scales, dq.scales)):
        a, b = a[1::2].contiguous(), b[1::2].contiguous()
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert torch.isnan(d.y[::2].float()).all()
    # gradients, and results written over inputs
    dx, _ = ops.rms_norm_rows_bwd(r, clean.sum, clean.rstd, w, dsum=x)
    ddx, _ = ops.rms_norm_rows_bwd(r, clean.sum, clean.rstd, w, dsum=dirty)
    assert torch.equal(dx[1::2], ddx[1::2])
    over = r.clone()
    y = torch.empty_like(x)
    ops.rms_norm_rows(x, w, over, out=ops.RmsNorm(y, None, over, None))
    assert torch.equal(y, clean.y) and torch.equal(over, clean.sum)
    over = x.clone()
    ops.rms_norm_rows_bwd(r, clean.sum, clean.rstd, w, dsum=over, grads=(over, torch.empty_like(w)))
    assert torch.equal(over, dx)


# ------------------------------------------------------------------ routing

def _ids(rng, T, k, E, bad=0.1, dtype=np.int32):
    ids = rng.integers(0, E, (T, k))
    ids[rng.random((T, k)) < bad] = -1
    return ids.astype(dtype)


def _check_sort(ids, E, **kw):
    T, k = ids.shape
    rows = torch.full((T * k,), -5, dtype=torch.int64, device="cuda")
    off = Guarded((E + 1,), torch.int64)
    slots = Guarded((T, k), torch.int32)
    r = ops.expert_sort(torch.from_numpy(ids).cuda(), E, out=ops.Routing(slots.t, off.t, rows), **kw)
    valid = np.where((ids >= 0) & (ids < E), ids, -1)
    # the same sort, vectorised: stable by expert
    flat = valid.reshape(-1)
    order = np.argsort(np.where(flat < 0, E, flat), kind="stable")
    n = int((flat >= 0).sum())
    ref = np.full(T * k, -1, np.int32)
    ref[order[:n]] = np.arange(n)
    assert np.array_equal(_np(r.slots), ref.reshape(T, k))
    assert np.array_equal(_np(r.offsets), np.concatenate([[0], np.cumsum(np.bincount(
        flat[flat >= 0], minlength=E))]))
    got = _np(rows)
    assert np.array_equal(got[:n], order[:n] // k) and (got[n:] == -5).all()
    off.check("offsets")
    slots.check("slots")
    return r


@pytest.mark.parametrize("T,k,E", [(0, 1, 4), (1, 1, 1), (1, 16, 3), (5, 2, 7), (31, 1, 64),
                                   (33, 3, 1000), (511, 2, 1024), (2048, 4, 64), (4096, 2, 512),
                                   (8191, 1, 2), (8193, 1, 1), (3000, 5, 60), (20000, 8, 256),
                                   (70001, 3, 1024), (300000, 2, 33)])
def test_sort(T, k, E):
    rng = np.random.default_rng(T + k + E)
    for dtype in (np.int32, np.int64):
        _check_sort(_ids(rng, T, k, E, dtype=dtype), E)
    if T:
        _check_sort(np.full((T, k), E - 1, np.int32), E)             # one expert takes all
        _check_sort(np.full((T, k), -1, np.int32), E)                # none takes any
        _check_sort(np.sort(_ids(rng, T, k, E), axis=0), E)          # sorted already


def test_sort_matches_the_oracle_and_reports_bad_ids():
    rng = np.random.default_rng(4)
    ids = _ids(rng, 50, 3, 9)
    r = _check_sort(ids, 9)
    slots, offsets, rows = ox.sort(ids, 9)
    assert np.array_equal(_np(r.slots), slots) and np.array_equal(_np(r.offsets), offsets)
    for T in (50, 20000):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        ids = _ids(rng, T, 3, 9)
        _check_sort(ids, 9, status=status)
        assert status.item() == 0
        ids[T // 2, 1], ids[T - 1, 2] = 9, 2 ** 31 - 1
        _check_sort(ids, 9, status=status)
        assert status.item() == ops.DEV_BAD_EXPERT


@pytest.mark.parametrize("width,dtype", [(1, torch.uint8), (3, torch.uint8), (16, torch.uint8),
                                         (100, torch.uint8), (7, BF), (64, BF), (1000, BF),
                                         (5000, BF), (6, F32), (1024, F32), (9, torch.int64)])
@pytest.mark.parametrize("T,k", [(1, 1), (5, 16), (130, 3)])
def test_dispatch(T, k, width, dtype):
    rng = np.random.default_rng(width + T)
    E = 5
    slots = ops.expert_sort(torch.from_numpy(_ids(rng, T, k, E, 0.2)).cuda(), E).slots
    x = torch.from_numpy(rng.integers(-100, 100, (T, width)) if dtype != torch.uint8
                         else rng.integers(0, 255, (T, width))).to(dtype).cuda()
    xs = ops.expert_dispatch(x, slots, out=torch.full((T * k, width), 77, device="cuda").to(dtype))
    ref = np.full((T * k, width), 77, np.float64)
    s = _np(slots)
    for t, j in np.argwhere(s >= 0):
        ref[s[t, j]] = _np(x)[t]
    assert np.array_equal(_np(xs).astype(np.float64), ref)
    # with scales, some places outside the buffer: those are skipped
    sc = _rand(3, T, 3, dtype=F32)
    most = max(1, T * k // 2)
    out, so = Guarded((most, width), dtype, 77), Guarded((most, 3), F32, 5.0)
    ops.expert_dispatch(x, slots, scales=sc, out=out.t, scales_out=so.t)
    ref_s = np.full((T * k, 3), 5.0)
    for t, j in np.argwhere(s >= 0):
        ref_s[s[t, j]] = _np(sc)[t]
    assert np.array_equal(_np(out.t).astype(np.float64), ref[:most])
    assert np.array_equal(_np(so.t), ref_s[:most])
    out.check("dispatch")
    so.check("dispatch scales")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("weights,residual", [(True, True), (False, False)])
@pytest.mark.parametrize("T,k,width", [(1, 1, 1), (3, 2, 7), (40, 5, 64), (33, 16, 100),
                                       (9, 8, 1000), (130, 3, 520), (5, 4, 4096), (2, 3, 9000)])
def test_combine_and_its_gradients(T, k, width, weights, residual, dtype):
    rng = np.random.default_rng(T + width)
    E = 6
    slots = ops.expert_sort(torch.from_numpy(_ids(rng, T, k, E, 0.2)).cuda(), E).slots
    y = _rand(1, T * k, width, dtype=dtype)
    named = np.zeros(T * k, bool)
    s = _np(slots)
    named[s[s >= 0]] = True
    y[torch.from_numpy(~named).cuda()] = float("nan")        # rows that nothing may read
    w = _rand(2, T, k, dtype=F32) if weights else None
    res = _rand(3, T, width, dtype=dtype) if residual else None
    out = Guarded((T, width), dtype)
    ops.expert_combine(y, slots, w, residual=res, out=out.t)
    ref = ox.combine(_np(y), s, _opt(w), _opt(res))
    size = ox.combine(np.abs(_np(y)), s, None if w is None else np.abs(_np(w)),
                      None if res is None else np.abs(_np(res)))
    _close(out.t, ref, np.abs(ref) * HALF[dtype] + (k + 2) * U * size, "combine")
    out.check("combine")
    do = _rand(4, T, width, dtype=dtype)
    dy, dw = Guarded((T * k, width), dtype, 7.0), Guarded((T, k), F32)
    ops.expert_combine_bwd(do, y, slots, w, grads=(dy.t, dw.t))
    rdy, rdw = ox.combine_bwd(_np(do), _np(y), s, _opt(w))
    rdy[~named] = 7.0                                        # left as they were
    _close(dy.t, rdy, np.abs(rdy) * (HALF[dtype] + U), "dy")
    size = ox.combine_bwd(np.abs(_np(do)), np.abs(_np(y)), s, None)[1]
    # a term's chain: up to 8 of each 256 columns (in 1 to 8 warps), 5 shuffles, 8 warps
    _close(dw.t, rdw, (8 * -(-width // 256) + 14) * U * size, "dweights")
    dy.check("dy")
    dw.check("dweights")
    # dy alone
    dy2 = Guarded((T * k, width), dtype, 7.0)
    ops.expert_combine_bwd(do, y, slots, w, grads=(dy2.t, None))
    assert torch.equal(dy2.t, dy.t)


def test_combine_skips_places_outside_and_dispatch_bwd_sums():
    slots = torch.tensor([[0, 9], [-1, 2 ** 31 - 1], [1, 0]], dtype=torch.int32, device="cuda")
    y = _rand(1, 2, 32, dtype=F32)
    out = ops.expert_combine(y, slots)
    assert torch.equal(out[0], y[0]) and not out[1].any()
    assert torch.equal(out[2], y[1] + y[0])                  # a row named twice may be read twice
    assert torch.equal(ops.expert_dispatch_bwd(y, slots), out)
    dw = ops.expert_combine_bwd(_rand(2, 3, 32, dtype=F32), y, slots, torch.ones(3, 2, device="cuda"))[1]
    assert dw[0, 1] == 0 and not dw[1].any()
    e = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    assert ops.expert_combine(y, e).shape == (0, 32)
    assert not ops.expert_combine(y[:0], slots).any()        # no rows at all
    for width in (7, 520):
        none = torch.empty(0, width, device="cuda")
        assert not ops.expert_combine(none, slots, torch.full((3, 2), float("nan"), device="cuda")).any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,k,width", [(700, 4, 1001), (5000, 3, 100), (90, 9, 2047), (3000, 2, 1024)])
def test_combine_over_its_residual_and_of_many_rows(T, k, width, dtype):
    """More tokens than blocks at once; the result written over the residual; rows that no slot
    names hold NaN."""
    rng = np.random.default_rng(T)
    r = ops.expert_sort(torch.from_numpy(_ids(rng, T, k, 16)).cuda(), 16)
    n = int(r.offsets[-1])
    y, res = _rand(1, T * k, width, dtype=dtype), _rand(2, T, width, dtype=dtype)
    y[n:] = float("nan")
    w = torch.rand(T, k, device="cuda")
    slots = r.slots.long()
    live = (slots >= 0).double()[..., None]
    rows = torch.nan_to_num(y.double()[slots.clamp_min(0)]) * live
    want = res.double() + (w.double()[..., None] * rows).sum(1)
    size = res.double().abs() + (w.double()[..., None] * rows.abs()).sum(1)
    out = res.clone()
    ops.expert_combine(y, r.slots, w, residual=out, out=out)
    _close(out, _np(want), _np(want.abs() * HALF[dtype] + size * (k + 1) * U), "over the residual")
    dout = _rand(3, T, width, dtype=dtype)
    dy, dw = ops.expert_combine_bwd(dout, y, r.slots, w)
    dots = (dout.double()[:, None, :] * rows).sum(2)
    mag = (dout.double()[:, None, :] * rows).abs().sum(2)
    _close(dw, _np(dots), _np(mag) * (width / 32 + 12) * U, "dweights")
    sorted_dy = (w.double()[..., None] * dout.double()[:, None, :])[slots >= 0]
    _close(dy[slots[slots >= 0]], _np(sorted_dy), _np(sorted_dy.abs()) * HALF[dtype] + 1e-40, "dy")


# ------------------------------------------------------------------ products

def _offsets(counts):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(counts)])).cuda()


COUNTS = [[1], [0, 5, 0], [128, 0, 129], [64, 65, 127, 1], [300, 3, 0, 0, 17],
          [0, 0, 0], [16, 17, 48, 49, 64, 0, 2], [1000, 24]]


def _dot_tol(K, size):
    return (K / 16 + 4) * 2.0 ** -22 * size


def _proj_case(counts, K, N, tail, seed):
    S, E = sum(counts) + tail, len(counts)
    x = _rand(seed, S, K) if S else torch.empty(0, K, dtype=BF, device="cuda")
    w = _rand(seed + 1, E, K, N, scale=K ** -0.5)
    off = _offsets(counts)
    if tail:
        x[S - tail:] = float("nan")              # rows of no expert must reach nothing
    return x, w, off, S, E


@pytest.mark.parametrize("K,N", [(8, 8), (64, 128), (72, 136), (200, 264), (256, 512), (1000, 40)])
@pytest.mark.parametrize("counts", COUNTS, ids=str)
def test_proj(counts, K, N):
    x, w, off, S, E = _proj_case(counts, K, N, 3, K + N + sum(counts))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ref = ox.proj(np.nan_to_num(_np(x)), _np(w), _np(off))
    size = ox.proj(np.nan_to_num(np.abs(_np(x))), np.abs(_np(w)), _np(off))
    live = S - 3
    for silu in (False, True):
        out, pre = Guarded((S, N), BF, 7.0), Guarded((S, N), BF, 7.0)
        ops.expert_proj(x, w, off, silu=silu, out=out.t, pre=pre.t if silu else None, status=status)
        want = ox.silu(ref) if silu else ref
        tol = np.abs(want) * (2 ** -8 + (2 ** -14 if silu else 0)) + 1.1 * _dot_tol(K, size) + 1e-30
        _close(out.t[:live], want[:live], tol[:live], "proj silu=%s" % silu)
        assert (out.t[live:] == 7).all()         # rows of no expert: left as they were
        out.check("proj")
        if silu:
            _close(pre.t[:live], ref[:live], (np.abs(ref) * 2 ** -8 + _dot_tol(K, size))[:live], "pre")
            assert (pre.t[live:] == 7).all()
            pre.check("pre")
    assert status.item() == 0


@pytest.mark.parametrize("K,N", [(16, 8), (128, 128), (144, 136), (400, 264), (512, 256)])
@pytest.mark.parametrize("counts", COUNTS, ids=str)
def test_proj_e4m3(counts, K, N):
    S, E = sum(counts) + 2, len(counts)
    g = torch.Generator().manual_seed(K + N)
    x = (torch.randn(S, K, generator=g) * 100).clamp(-448, 448).to(ops.F8).cuda()
    w = (torch.randn(E, N, K, generator=g) * 100).clamp(-448, 448).to(ops.F8).cuda()
    xs = (torch.rand(S, generator=g) * 0.01).cuda()
    ws = (torch.rand(E, N, generator=g) * 0.01).cuda()
    off = _offsets(counts)
    a, b = _np(x) * _np(xs)[:, None], np.swapaxes(_np(w) * _np(ws)[..., None], 1, 2)
    ref, size = ox.proj(a, b, _np(off)), ox.proj(np.abs(a), np.abs(b), _np(off))
    for silu in (False, True):
        out = Guarded((S, N), BF, 7.0)
        ops.expert_proj_e4m3(x, xs if silu else xs[:, None], w, ws, off, silu=silu, out=out.t)
        want = ox.silu(ref) if silu else ref
        tol = np.abs(want) * (2 ** -8 + (2 ** -14 if silu else 0)) + 1.1 * (
            _dot_tol(K, size) + 3 * U * np.abs(ref)) + 1e-30
        _close(out.t[:S - 2], want[:S - 2], tol[:S - 2], "e4m3 silu=%s" % silu)
        assert (out.t[S - 2:] == 7).all()
        out.check("proj e4m3")


@pytest.mark.parametrize("K,N", [(8, 8), (64, 128), (136, 72), (264, 200), (256, 512), (40, 1000)])
@pytest.mark.parametrize("counts", COUNTS, ids=str)
def test_proj_bwd(counts, K, N):
    x, w, off, S, E = _proj_case(counts, K, N, 3, K + N + sum(counts))
    live = S - 3
    do = _rand(9, S, N)
    do[live:] = float("nan")
    pre = _rand(10, S, K, scale=2.0)
    X, D = np.nan_to_num(_np(x)), np.nan_to_num(_np(do))
    X[live:] = 0
    for p in (None, pre):
        gx, gw = Guarded((S, K), BF, 7.0), Guarded((E, K, N), BF, 7.0)
        ops.expert_proj_bwd(do, x, w, off, silu_pre=p, grads=(gx.t, gw.t))
        rdx, rdw = ox.proj_bwd(D, X, _np(w), _np(off), _opt(p))
        sdx, sdw = ox.proj_bwd(np.abs(D), np.abs(X), np.abs(_np(w)), _np(off))
        tol = np.abs(rdx) * (2 ** -8 + (0 if p is None else 2 ** -14)) + 1.1 * _dot_tol(N, sdx)
        _close(gx.t[:live], rdx[:live], tol[:live] + 1e-30, "dx")
        assert (gx.t[live:] == 7).all()
        _close(gw.t, rdw, np.abs(rdw) * 2 ** -8 + _dot_tol(max(counts), sdw), "dw")
        gx.check("dx")
        gw.check("dw")
        # one gradient alone
        one = ops.expert_proj_bwd(do, x, w, off, silu_pre=p, grads=(torch.empty_like(x), None))
        assert torch.equal(one[0][:live], gx.t[:live])
        one = ops.expert_proj_bwd(do, x, w, off, grads=(None, torch.empty_like(w)))
        assert torch.equal(one[1], gw.t)


@pytest.mark.parametrize("counts,K,N", [([399, 1], 72, 6400), ([130, 257, 600, 2, 63], 200, 3336),
                                        ([1, 0, 63, 64, 65, 127, 129, 300, 2, 5000], 520, 1032),
                                        ([700, 2, 0, 5300, 3001, 63], 1032, 512),
                                        ([9000, 1100], 512, 2056)],
                         ids=["wide", "ragged", "rows", "narrow", "long"])
def test_products_large_enough_for_pairs_of_blocks(counts, K, N):
    """Few and many rows per expert where the products run on pairs of blocks (256 x 256 tiles):
    rows of no expert hold NaN, and short last slices of the weight gradients' contraction."""
    x, w, off, S, E = _proj_case(counts, K, N, 3, K + N)
    live = S - 3
    do, pre = _rand(9, S, N), _rand(10, S, K)
    do[live:] = float("nan")
    out, p = Guarded((S, N), BF, 7.0), Guarded((S, N), BF, 7.0)
    gx, gw = Guarded((S, K), BF, 7.0), Guarded((E, K, N), BF)
    ops.expert_proj(x, w, off, silu=True, out=out.t, pre=p.t)
    ops.expert_proj_bwd(do, x, w, off, silu_pre=pre, grads=(gx.t, gw.t))
    for e, (a, b) in enumerate(zip(_np(off), _np(off)[1:])):
        X, W, D = x[a:b].double(), w[e].double(), do[a:b].double()
        q = pre[a:b].double()
        slope = torch.sigmoid(q) * (1 + q * torch.sigmoid(-q))
        r = X @ W
        dot = _dot_tol(K, X.abs() @ W.abs())
        for got, ref, tol in (
                (p.t[a:b], r, r.abs() * 2 ** -8 + dot),
                (out.t[a:b], r * torch.sigmoid(r), (r * torch.sigmoid(r)).abs() * (2 ** -8 + 2 ** -14)
                 + 1.1 * dot),
                (gx.t[a:b], (D @ W.T) * slope, ((D @ W.T) * slope).abs() * (2 ** -8 + 2 ** -14)
                 + 1.1 * _dot_tol(N, D.abs() @ W.T.abs())),
                (gw.t[e], X.T @ D, (X.T @ D).abs() * 2 ** -8 + _dot_tol(int(b - a), X.T.abs() @ D.abs()))):
            assert ((got.double() - ref).abs() <= tol + 1e-30).all(), e
    for g, rows in ((out, live), (p, live), (gx, live)):
        assert (g.t[rows:] == 7).all()
    for g in (out, p, gx, gw):
        g.check("pairs")
    if K % 16 == 0 or K == 200:
        K8 = K // 16 * 16
        xq = (x[:, :K8].float() * 50).nan_to_num().clamp(-448, 448).to(ops.F8).contiguous()
        wq = (w.float().transpose(1, 2) * 200)[:, :, :K8].clamp(-448, 448).to(ops.F8).contiguous()
        xs, ws = torch.rand(S, device="cuda") * 0.02, torch.rand(E, N, device="cuda") * 0.005
        out = Guarded((S, N), BF, 7.0)
        ops.expert_proj_e4m3(xq, xs, wq, ws, off, out=out.t)
        for e, (a, b) in enumerate(zip(_np(off), _np(off)[1:])):
            X = xq[a:b].double() * xs[a:b, None].double()
            W = (wq[e].double() * ws[e][:, None].double()).T
            r = X @ W
            tol = r.abs() * (2 ** -8 + 3 * U) + _dot_tol(K8, X.abs() @ W.abs())
            assert ((out.t[a:b].double() - r).abs() <= tol + 1e-30).all(), e
        assert (out.t[live:] == 7).all()
        out.check("pairs e4m3")


@pytest.mark.parametrize("counts,K,N", [([5000], 64, 128), ([3000, 0, 2003], 72, 136),
                                        ([20, 9000, 65], 256, 200), ([1100, 1029], 512, 264)],
                         ids=str)
def test_weight_gradients_from_parts_of_the_rows(counts, K, N):
    """Few small matrices and many rows: the contraction is cut into parts that are added up."""
    x, w, off, S, E = _proj_case(counts, K, N, 3, K + N)
    do = _rand(9, S, N)
    do[S - 3:] = float("nan")
    gw = Guarded((E, K, N), BF)
    ops.expert_proj_bwd(do, x, w, off, grads=(None, gw.t))
    for e, (a, b) in enumerate(zip(_np(off), _np(off)[1:])):
        X, D = x[a:b].double(), do[a:b].double()
        tol = (X.T @ D).abs() * 2 ** -8 + _dot_tol(int(b - a), X.T.abs() @ D.abs()) + 1e-30
        assert ((gw.t[e].double() - X.T @ D).abs() <= tol).all(), e
    gw.check("dw")
    again = ops.expert_proj_bwd(do, x, w, off, grads=(None, torch.empty_like(w)))[1]
    assert torch.equal(again, gw.t)


# few tiles and long contractions: several blocks share a tile, each a part of the contraction
@pytest.mark.parametrize("counts", [[1], [0, 3, 0, 130], [64, 65], [128, 7, 1, 0, 127], [2] * 7], ids=str)
@pytest.mark.parametrize("K,N", [(1024, 64), (2048, 136), (520, 264), (1032, 72), (4104, 8), (264, 128)])
def test_products_whose_contraction_is_shared(counts, K, N):
    test_proj(counts, K, N)
    test_proj_e4m3(counts, -(-K // 16) * 16, N)
    test_proj_bwd(counts, N, K)


def test_shared_contractions_repeat_and_cover_overlapping_experts():
    x, w, _, S, _ = _proj_case([4990, 0, 0, 10], 512, 64, 0, 8)
    off = torch.tensor([0, 4990, 0, 4990, 5000], dtype=torch.int64, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = ops.expert_proj(x, w, off, status=status)
    assert status.item() == ops.DEV_BAD_OFFSETS              # expert 1 ends ahead of its start
    ref = ox.proj(_np(x[4990:]), _np(w[3:]), np.array([0, 10]))
    size = ox.proj(np.abs(_np(x[4990:])), np.abs(_np(w[3:])), np.array([0, 10]))
    _close(out[4990:], ref, np.abs(ref) * 2 ** -8 + _dot_tol(512, size), "behind the overlap")
    x, w, off, S, E = _proj_case([64, 65], 4104, 136, 0, 9)
    first = ops.expert_proj(x, w, off, silu=True)
    for _ in range(5):
        assert torch.equal(ops.expert_proj(x, w, off, silu=True), first)


def test_proj_without_rows():
    x, w, off, _, _ = _proj_case([0, 0], 64, 64, 0, 1)
    assert ops.expert_proj(x, w, off).shape == (0, 64)
    dx, dw = ops.expert_proj_bwd(torch.empty(0, 64, dtype=BF, device="cuda"), x, w, off)
    assert dx.shape == (0, 64) and not dw.any()


def test_proj_reports_bad_offsets_and_skips_their_experts():
    x, w, _, S, _ = _proj_case([40, 40, 40], 64, 64, 0, 2)
    for off, good in (([0, 40, 30, 120], (0, 2)), ([0, 40, 121, 120], (0,)),
                      ([-1, 40, 80, 120], (1, 2)), ([5, 40, 80, 100], (0, 1, 2)),
                      ([0, 2 ** 40, 80, 120], (2,))):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        o = torch.tensor(off, dtype=torch.int64, device="cuda")
        out = torch.full((S, 64), 7.0, dtype=BF, device="cuda")
        ops.expert_proj(x, w, o, out=out, status=status)
        assert status.item() == (0 if len(good) == 3 else ops.DEV_BAD_OFFSETS), off
        dw = ops.expert_proj_bwd(out, x, w, o)[1]
        touched = np.zeros(S, bool)
        for e in good:
            touched[off[e]:off[e + 1]] = True
        assert (out[torch.from_numpy(~touched).cuda()] == 7).all()
        for e in range(3):
            if e not in good:
                assert not dw[e].any()


def test_many_experts_and_large_products():
    """1024 experts of which few have rows; a product of several waves of wide tiles."""
    counts = np.zeros(1024, np.int64)
    counts[[0, 1, 511, 512, 1023]] = [3, 200, 1, 130, 64]
    x, w, off, S, E = _proj_case(list(counts), 64, 136, 1, 3)
    out = ops.expert_proj(x, w, off)
    ref = ox.proj(np.nan_to_num(_np(x)), _np(w), _np(off))
    size = ox.proj(np.nan_to_num(np.abs(_np(x))), np.abs(_np(w)), _np(off))
    _close(out[:S - 1], ref[:S - 1], (np.abs(ref) * 2 ** -8 + _dot_tol(64, size))[:S - 1], "1024")
    counts = [3000, 0, 5001, 129, 2000]
    x, w, off, S, E = _proj_case(counts, 512, 1032, 0, 4)
    do = _rand(5, S, 1032)
    out = ops.expert_proj(x, w, off)
    dx, dw = ops.expert_proj_bwd(do, x, w, off)
    # the same formulas in fp64 on the GPU (elementary products), for the size
    for e, (a, b) in enumerate(zip(_np(off), _np(off)[1:])):
        X, W, D = x[a:b].double(), w[e].double(), do[a:b].double()
        for got, p, q in ((out[a:b], X, W), (dx[a:b], D, W.T), (dw[e], X.T, D)):
            r = p @ q
            tol = r.abs() * 2 ** -8 + _dot_tol(p.shape[1], p.abs() @ q.abs())
            assert ((got.double() - r).abs() <= tol).all()


def test_tensors_of_more_than_two_to_the_31_elements():
    """Rows whose element offsets pass 32 bits, at both ends of every operator."""
    S, W, E = 270_000, 8192, 2                       # 2.2e9 elements, 4.4 GB in bf16
    x = torch.zeros(S, W, dtype=BF, device="cuda")
    ends = [0, 1, S - 2, S - 1]
    part = _rand(1, 4, W)
    x[ends] = part
    r = ops.rms_norm_rows(x, e4m3=True, group=128)
    small = ops.rms_norm_rows(part, e4m3=True, group=128)
    assert torch.equal(r.y[ends].view(torch.uint8), small.y.view(torch.uint8))
    assert torch.equal(r.scales[ends], small.scales) and not r.y[5].float().any()
    del r
    slots = torch.tensor([[S - 1, 0], [1, S - 2]], dtype=torch.int32, device="cuda")
    out = ops.expert_combine(x, slots)
    assert torch.equal(out, (torch.stack([part[3].float() + part[0].float(),
                                          part[1].float() + part[2].float()])).to(BF))
    w = _rand(2, E, W, 64, scale=W ** -0.5)
    off = torch.tensor([0, S - 1, S], device="cuda")
    y = ops.expert_proj(x, w, off)
    # (each on its own: few rows share the contraction among blocks, so the sums' order differs)
    few = np.array([0, 3, 4])
    ref, size = ox.proj(_np(part), _np(w), few), ox.proj(np.abs(_np(part)), np.abs(_np(w)), few)
    for got in (y[ends], ops.expert_proj(part, w, torch.from_numpy(few).cuda())):
        _close(got, ref, np.abs(ref) * 2 ** -8 + _dot_tol(W, size), "ends")
    xs = ops.expert_dispatch(part[:2], slots, out=x)
    assert torch.equal(xs[ends], torch.stack([part[0], part[1], part[1], part[0]]))


# ------------------------------------------------------------------ the layer

def _layer_case(T, k, E, d, ff, seed):
    rng = np.random.default_rng(seed)
    x, res = _rand(seed, T, d), _rand(seed + 1, T, d, scale=2.0)
    nw = 1 + 0.1 * _rand(seed + 2, d, dtype=F32)
    ids = torch.from_numpy(_ids(rng, T, k, E)).cuda()
    gates = torch.softmax(_rand(seed + 3, T, k, dtype=F32), 1)
    w_in, w_out = _rand(seed + 4, E, d, ff, scale=d ** -0.5), _rand(seed + 5, E, ff, d, scale=ff ** -0.5)
    return x, res, nw, ids, gates, w_in, w_out


def _rel(got, ref):
    return float(np.linalg.norm(_np(got) - ref) / np.linalg.norm(ref))


@pytest.mark.parametrize("T,k,E,d,ff", [(1, 1, 1, 64, 64), (300, 2, 8, 128, 256), (77, 3, 5, 72, 136)])
def test_layer_forward_and_gradients(T, k, E, d, ff):
    """The operators together.  Each tensor that passes between them is rounded to bf16 (2^-8 of a
    value at most); a random product carries a relative error on with a factor of at most 2, so
    an output behind n roundings is within 2 n 2^-8 of its 2-norm: n = 4 forward, 8 backward."""
    x, res, nw, ids, gates, w_in, w_out = _layer_case(T, k, E, d, ff, T)
    s = ops.expert_layer_fwd(x, res, nw, ids, gates, w_in, w_out, training=True)
    ref = ox.layer(_np(x), _np(res), _np(nw), _np(ids), _np(gates), _np(w_in), _np(w_out), 1e-5)
    assert np.array_equal(_np(s["routing"].slots), ref["slots"])
    assert _rel(s["o"].float() - s["sum"].float(), ref["o"] - ref["h"]) < 8 * 2 ** -8 + \
        2 ** -8 * np.linalg.norm(ref["o"]) / max(np.linalg.norm(ref["o"] - ref["h"]), 1e-9)
    do = _rand(99, T, d)
    g = ops.expert_layer_bwd(do, s, nw, gates, w_in, w_out)
    want = ox.layer_bwd(_np(do), ref, _np(nw), _np(gates), _np(w_in), _np(w_out))
    for name, r in want.items():
        assert _rel(g[name], r) < 16 * 2 ** -8, name
    # inference gives the same output
    o = ops.expert_layer_fwd(x, res, nw, ids, gates, w_in, w_out)["o"]
    assert torch.equal(o, s["o"])


def test_layer_with_the_8_bit_product():
    """As above, with the norm's output and w_in in e4m3: 2^-4 of a value at most each."""
    x, res, nw, ids, gates, w_in, w_out = _layer_case(300, 2, 8, 128, 256, 3)
    wt = w_in.float().transpose(1, 2).contiguous()
    ws = (wt.abs().amax(2) / 448).contiguous()
    wq = (wt / ws[..., None]).clamp(-448, 448).to(ops.F8)
    s = ops.expert_layer_fwd(x, res, nw, ids, gates, (wq, ws), w_out)
    ref = ox.layer(_np(x), _np(res), _np(nw), _np(ids), _np(gates), _np(w_in), _np(w_out), 1e-5)
    assert _rel(s["o"].float() - s["sum"].float(), ref["o"] - ref["h"]) < 2 * (2 * 2 ** -4)


def test_layer_on_a_stream_and_in_a_graph():
    """On another stream and captured: the same bits, also after the inputs changed in place."""
    a = _layer_case(200, 2, 6, 128, 128, 8)
    do = _rand(5, 200, 128)

    def step(stream=None):
        s = ops.expert_layer_fwd(*a, training=True, stream=stream)
        g = ops.expert_layer_bwd(do, s, a[2], a[4], a[5], a[6], stream=stream)
        return [s["o"]] + [g[n] for n in sorted(g)]

    ref = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for p, q in zip(step(side), ref):
        side.synchronize()
        assert torch.equal(p, q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    torch.cuda.synchronize()
    for p, q in zip(got, ref):
        assert torch.equal(p, q)
    b = _layer_case(200, 2, 6, 128, 128, 21)
    for p, q in zip(a, b):
        p.copy_(q)
    graph.replay()
    torch.cuda.synchronize()
    for p, q in zip(got, step()):
        assert torch.equal(p, q)


def test_two_streams_at_once():
    """Two layers in flight at the same time, with workspaces of their own."""
    cases = [_layer_case(9000, 2, 16, 128, 128, s) for s in (1, 2)]
    refs = [ops.expert_layer_fwd(*c)["o"] for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[], []]
    for _ in range(4):
        for i, (c, st) in enumerate(zip(cases, streams)):
            outs[i].append(ops.expert_layer_fwd(*c, stream=st)["o"])
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            assert torch.equal(o, refs[i])


def test_a_wait_that_runs_out_is_reported():
    """A planted wait that nothing satisfies runs out after a millisecond: the products say so and
    leave the GPU usable; the next call is right again."""
    x, w, off, S, E = _proj_case([300, 200], 512, 256, 0, 6)
    ref = ops.expert_proj(x, w, off)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.set_wait_test(2_000_000, True)
    try:
        ops.expert_proj(x, w, off, status=status)
        torch.cuda.synchronize()
    finally:
        ops.set_wait_test(0, False)
    assert status.item() == ops.DEV_WAIT_TIMEOUT
    status.zero_()
    assert torch.equal(ops.expert_proj(x, w, off, status=status), ref) and status.item() == 0
