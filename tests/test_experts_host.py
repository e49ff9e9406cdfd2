"""The mixture-of-experts operators without a GPU: the fp64 oracle's gradients against central
differences and hand-worked routing, and every refusal of the C ABI and of its binding, which
come before anything is enqueued."""
import ctypes

import numpy as np
import pytest
import torch

from jagged_hstu_attention_02_b200 import ops
from oracle import experts as ox

INVALID, UNSUPPORTED, TOO_SMALL = 1, 2, 3


def _differences(f, a, step=1e-5):
    g = np.zeros(a.shape)
    for i in np.ndindex(*a.shape):
        keep = a[i]
        a[i] = keep + step
        up = f()
        a[i] = keep - step
        down = f()
        a[i] = keep
        g[i] = (up - down) / (2 * step)
    return g


def test_oracle_layer_gradients_match_differences():
    rng = np.random.default_rng(5)
    T, k, E, d, ff = 5, 2, 3, 4, 6
    x, res = rng.standard_normal((T, d)), rng.standard_normal((T, d))
    nw = 1 + 0.1 * rng.standard_normal(d)
    ids = np.array([[0, 2], [2, 0], [-1, -1], [0, -1], [2, 2]], np.int32)   # expert 1: no rows
    gates = rng.random((T, k))
    w_in, w_out = rng.standard_normal((E, d, ff)), rng.standard_normal((E, ff, d))
    do = rng.standard_normal((T, d))

    def loss():
        return float((ox.layer(x, res, nw, ids, gates, w_in, w_out, 1e-5)["o"] * do).sum())

    s = ox.layer(x, res, nw, ids, gates, w_in, w_out, 1e-5)
    g = ox.layer_bwd(do, s, nw, gates, w_in, w_out)
    gates_ref = _differences(loss, gates)
    for got, ref in ((g["dx"], _differences(loss, x)), (g["dx"], _differences(loss, res)),
                     (g["dnorm_weight"], _differences(loss, nw)), (g["dgates"], gates_ref),
                     (g["dw_in"], _differences(loss, w_in)),
                     (g["dw_out"], _differences(loss, w_out))):
        # central differences: error ~ step^2 * f''' (1e-10 * O(10)) + 1e-16 / step * O(10)
        np.testing.assert_allclose(got, ref, rtol=0, atol=2e-8 * max(1, np.abs(ref).max()) + 2e-8)
    assert not g["dw_in"][1].any() and not g["dgates"][2].any()


def test_oracle_sort_on_a_hand_worked_example():
    ids = np.array([[1, 0], [-1, 1], [1, 3]], np.int32)
    slots, offsets, rows = ox.sort(ids, 4)
    assert slots.tolist() == [[1, 0], [-1, 2], [3, 4]]
    assert offsets.tolist() == [0, 1, 4, 4, 5]
    assert rows.tolist() == [0, 0, 1, 2, 2]


def _p(x=0x1000):
    return ctypes.c_void_p(x)


def test_norm_refusals():
    L = ops.lib()
    mis = _p(0x1008)

    def fwd(x=_p(), res=None, w=None, rows=4, width=64, eps=1e-5, dt=ops.HSTU_BF16, y=_p(),
            s=None, r=None):
        return L.hstu_rms_norm_rows(x, res, w, rows, width, eps, dt, y, s, r, None)

    for bad in (dict(x=None), dict(y=None), dict(rows=-1), dict(rows=2 ** 31), dict(width=0),
                dict(width=16385), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(dt=2), dict(x=mis), dict(res=mis), dict(w=mis),
                dict(y=mis), dict(s=mis), dict(r=mis)):
        assert fwd(**bad) == INVALID, bad
    assert fwd(rows=0) == 0                      # nothing to do: nothing is enqueued

    def q(group=0, scales=_p()):
        return L.hstu_rms_norm_rows_e4m3(_p(), None, None, 4, 64, 1e-5, ops.HSTU_BF16, group, _p(),
                                         scales, None, None, None)

    for bad in (dict(group=16), dict(group=-1), dict(group=256), dict(scales=None)):
        assert q(**bad) == INVALID, bad

    n = ctypes.c_size_t()
    assert L.hstu_rms_norm_rows_bwd_workspace_size(4, 64, None) == INVALID
    assert L.hstu_rms_norm_rows_bwd_workspace_size(4, 0, ctypes.byref(n)) == INVALID
    assert L.hstu_rms_norm_rows_bwd_workspace_size(100, 64, ctypes.byref(n)) == 0

    def bwd(dy=_p(), h=_p(), r=_p(), dx=_p(), dw=_p(), ws=_p(), nb=n.value, rows=100, dt=1):
        return L.hstu_rms_norm_rows_bwd(dy, h, r, None, None, rows, 64, dt, dx, dw, ws, nb, None)

    for bad in (dict(dy=None), dict(h=None), dict(r=None), dict(dx=None), dict(ws=None),
                dict(rows=-1), dict(dt=9), dict(dx=mis), dict(ws=mis)):
        assert bwd(**bad) == INVALID, bad
    assert bwd(nb=n.value - 1) == TOO_SMALL


def test_routing_refusals():
    L = ops.lib()
    n = ctypes.c_size_t()
    size = L.hstu_expert_sort_workspace_size
    for T, k, E in ((-1, 1, 4), (4, 0, 4), (4, 17, 4), (2 ** 31, 1, 4), (2 ** 28, 16, 4),
                    (4, 1, 0), (4, 1, 1025)):
        assert size(T, k, E, ctypes.byref(n)) == INVALID, (T, k, E)
    assert size(4, 1, 4, None) == INVALID
    assert size(4, 2, 4, ctypes.byref(n)) == 0 and n.value == 0
    assert size(1 << 20, 2, 64, ctypes.byref(n)) == 0 and n.value > 0
    need = n.value

    def sort(ids=_p(), w64=0, T=1 << 20, k=2, E=64, slots=_p(), off=_p(), rows=None, ws=_p(),
             nb=need):
        return L.hstu_expert_sort(ids, w64, T, k, E, slots, off, rows, None, ws, nb, None)

    for bad in (dict(ids=None), dict(w64=2), dict(slots=None), dict(off=None), dict(ws=None),
                dict(ids=_p(8)), dict(off=_p(8)), dict(k=0), dict(E=0)):
        assert sort(**bad) == INVALID, bad
    assert sort(nb=need - 1) == TOO_SMALL

    def disp(x=_p(), rb=64, sc=None, ns=0, slots=_p(), T=4, k=2, mr=8, out=_p(), so=None):
        return L.hstu_expert_dispatch(x, rb, sc, ns, slots, T, k, mr, out, so, None)

    for bad in (dict(x=None), dict(rb=0), dict(slots=None), dict(T=-1), dict(k=17), dict(mr=-1),
                dict(out=None), dict(sc=_p(), ns=1), dict(sc=_p(), ns=0, so=_p()), dict(so=_p()),
                dict(x=_p(8)), dict(out=_p(8))):
        assert disp(**bad) == INVALID, bad
    assert disp(T=0) == 0 and disp(mr=0) == 0

    def comb(y=_p(), slots=_p(), w=None, res=None, T=4, k=2, mr=8, width=32, dt=1, out=_p()):
        return L.hstu_expert_combine(y, slots, w, res, T, k, mr, width, dt, out, None)

    for bad in (dict(y=None), dict(slots=None), dict(T=-1), dict(k=0), dict(mr=-1), dict(width=0),
                dict(dt=3), dict(out=None), dict(y=_p(4)), dict(res=_p(4)), dict(w=_p(4))):
        assert comb(**bad) == INVALID, bad
    assert comb(T=0) == 0

    def cbwd(do=_p(), y=_p(), slots=_p(), mr=8, dt=1, dy=_p(), dw=_p(), width=32):
        return L.hstu_expert_combine_bwd(do, y, slots, None, 4, 2, mr, width, dt, dy, dw, None)

    for bad in (dict(do=None), dict(y=None), dict(slots=None), dict(mr=-1), dict(dt=2),
                dict(dy=None), dict(dw=_p(4)), dict(width=-8)):
        assert cbwd(**bad) == INVALID, bad


def test_combine_refuses_rows_whose_counters_would_overflow():
    L = ops.lib()
    for width in (2 ** 30 + 1, 2 ** 31 - 1):
        assert L.hstu_expert_combine(_p(), _p(), None, None, 4, 2, 8, width, 1, _p(), None) == INVALID
        assert L.hstu_expert_combine_bwd(_p(), _p(), _p(), None, 4, 2, 8, width, 1, _p(), None, None) == INVALID


def test_product_refusals():
    L = ops.lib()

    def fwd(x=_p(), w=_p(), off=_p(), S=4, E=2, K=64, N=64, silu=0, out=_p(), pre=None):
        return L.hstu_expert_proj(x, w, off, S, E, K, N, silu, out, pre, None, None)

    for bad in (dict(x=None), dict(w=None), dict(off=None), dict(S=-1), dict(S=2 ** 31),
                dict(E=0), dict(E=1025), dict(K=0), dict(K=12), dict(K=65544), dict(N=4),
                dict(N=0), dict(N=65544), dict(silu=2), dict(out=None), dict(pre=_p()),
                dict(x=_p(8)), dict(w=_p(8)), dict(out=_p(8))):
        assert fwd(**bad) == INVALID, bad
    assert fwd(S=0) == 0

    def q(xs=_p(), ws=_p(), K=64, N=64):
        return L.hstu_expert_proj_e4m3(_p(), xs, _p(), ws, _p(), 4, 2, K, N, 0, _p(), None, None)

    for bad in (dict(xs=None), dict(ws=None), dict(K=8), dict(K=72), dict(N=12), dict(ws=_p(8))):
        assert q(**bad) == INVALID, bad

    n = ctypes.c_size_t()
    size = L.hstu_expert_proj_bwd_workspace_size
    assert size(4, 2, 64, 64, None) == INVALID and size(4, 0, 64, 64, ctypes.byref(n)) == INVALID
    assert size(4, 2, 64, 64, ctypes.byref(n)) == 0 and n.value == 0
    assert size(30000, 2, 64, 64, ctypes.byref(n)) == 0 and n.value > 0
    need = n.value

    def bwd(do=_p(), x=_p(), w=_p(), off=_p(), S=4, K=64, N=64, dx=_p(), dw=_p(), ws=None, nb=0):
        return L.hstu_expert_proj_bwd(do, x, w, off, None, S, 2, K, N, dx, dw, None, ws, nb, None)

    assert bwd(S=30000) == INVALID and bwd(S=30000, ws=_p(8), nb=need) == INVALID
    assert bwd(S=30000, ws=_p(), nb=need - 1) == TOO_SMALL

    for bad in (dict(do=None), dict(x=None), dict(w=None), dict(off=None), dict(S=-1),
                dict(K=20), dict(N=20), dict(dx=_p(8)), dict(dw=_p(8))):
        assert bwd(**bad) == INVALID, bad
    assert bwd(dx=None, dw=None, x=None, w=None) == 0


def test_binding_refuses_wrong_shapes_types_and_places():
    bf, f32 = torch.bfloat16, torch.float32
    x = torch.zeros(4, 16, dtype=bf)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    off = torch.zeros(3, dtype=torch.int64)
    w = torch.zeros(2, 16, 8, dtype=bf)
    xs = torch.zeros(8, 16, dtype=bf)
    calls = [
        lambda: ops.rms_norm_rows(x),                                        # not on a GPU
        lambda: ops.rms_norm_rows(x.half()),
        lambda: ops.rms_norm_rows(x[0]),
        lambda: ops.rms_norm_rows(x, group=32),
        lambda: ops.rms_norm_rows(x, e4m3=True, group=16),
        lambda: ops.rms_norm_rows(x, torch.zeros(16, dtype=bf)),
        lambda: ops.rms_norm_rows(x, torch.zeros(8)),
        lambda: ops.rms_norm_rows(x, residual=x[:2]),
        lambda: ops.rms_norm_rows(x, residual=x.float()),
        lambda: ops.rms_norm_rows_bwd(x, x, torch.zeros(3)),
        lambda: ops.rms_norm_rows_bwd(x, x.float(), torch.zeros(4)),
        lambda: ops.expert_sort(ids, 2),
        lambda: ops.expert_sort(ids[0], 2),
        lambda: ops.expert_sort(ids.to(torch.int16), 2),
        lambda: ops.expert_sort(ids, 2, status=torch.zeros(1)),
        lambda: ops.expert_dispatch(x, ids),
        lambda: ops.expert_dispatch(x[:3], ids),
        lambda: ops.expert_dispatch(x, ids.long()),
        lambda: ops.expert_dispatch(x, ids, scales=torch.zeros(4)),
        lambda: ops.expert_dispatch(x, ids, scales_out=torch.zeros(8, 1)),
        lambda: ops.expert_combine(xs, ids, torch.zeros(4, 2, dtype=bf)),
        lambda: ops.expert_combine(xs, ids, torch.zeros(4, 3)),
        lambda: ops.expert_combine(xs, ids, residual=x[:, :8]),
        lambda: ops.expert_combine_bwd(x.float(), xs, ids),
        lambda: ops.expert_proj(xs, w, off),
        lambda: ops.expert_proj(xs.float(), w, off),
        lambda: ops.expert_proj(xs, w[:, :8], off),
        lambda: ops.expert_proj(xs, w, off[:2]),
        lambda: ops.expert_proj(xs, w, off.int()),
        lambda: ops.expert_proj_e4m3(xs, torch.zeros(8), w, torch.zeros(2, 8), off),
        lambda: ops.expert_proj_bwd(xs, xs, w, off),
        lambda: ops.expert_proj_bwd(torch.zeros(8, 8, dtype=f32), xs, w, off),
        lambda: ops.expert_layer_fwd(x, None, None, ids, None, (w, w), w, training=True),
    ]
    for c in calls:
        with pytest.raises(ValueError):
            c()


def test_binding_refuses_sizes_that_the_c_abi_would_cut_to_32_bits():
    """2^32 + 64 columns are not 64: the tensors have no memory, and the size is refused first."""
    wide, bf = 2 ** 32 + 64, torch.bfloat16

    def empty(*shape, dtype=bf):
        return torch.empty(*shape, dtype=dtype, device="meta")

    one = empty(1, 1, dtype=torch.int32)
    off, scale = empty(2, dtype=torch.int64), empty(1, dtype=torch.float32)
    calls = [
        lambda: ops.rms_norm_rows(empty(1, wide)),
        lambda: ops.rms_norm_rows(empty(1, wide), e4m3=True, group=128),
        lambda: ops.rms_norm_rows_bwd(empty(1, wide), empty(1, wide), scale),
        lambda: ops.expert_sort(one, wide),
        lambda: ops.expert_sort(empty(1, wide, dtype=torch.int32), 4),
        lambda: ops.expert_dispatch(empty(1, 64), empty(1, wide, dtype=torch.int32)),
        lambda: ops.expert_dispatch(empty(1, 64), one, scales=empty(1, wide, dtype=torch.float32)),
        lambda: ops.expert_combine(empty(1, wide), one),
        lambda: ops.expert_combine_bwd(empty(1, wide), empty(1, wide), one),
        lambda: ops.expert_proj(empty(1, wide), empty(1, wide, 8), off),
        lambda: ops.expert_proj(empty(1, 8), empty(1, 8, wide), off),
        lambda: ops.expert_proj(empty(1, 8), empty(wide, 8, 8), empty(wide + 1, dtype=torch.int64)),
        lambda: ops.expert_proj_e4m3(empty(1, wide, dtype=ops.F8), scale, empty(1, 8, wide, dtype=ops.F8),
                                     empty(1, 8, dtype=torch.float32), off),
        lambda: ops.expert_proj_bwd(empty(1, 8), empty(1, wide), empty(1, wide, 8), off),
    ]
    for c in calls:
        with pytest.raises(ValueError, match="2.31 or more"):
            c()


def test_products_refuse_sizes_whose_tiles_could_pass_32_bits():
    """Offsets 0, rows, 0, rows, ... give every second expert all rows.  The kernels reject the
    experts between and count the others' tiles in 32 bits: 1024 experts, 2^30 rows of one column
    of tiles would be 2^32, which is 0 tiles or places outside of the tensors."""
    L = ops.lib()

    def tiles(rows, E, cols):                          # as the kernels' table adds them up
        return sum(-(-rows // 128) for e in range(E) if e % 2 == 0) * -(-cols // 128)

    for rows, E, cols in ((2 ** 30, 1024, 8), (2 ** 22, 1024, 65536), (2 ** 31 - 1, 511, 128),
                          (2 ** 25, 1023, 4096)):
        assert tiles(rows, E, cols) >= 2 ** 31
        assert L.hstu_expert_proj(_p(), _p(), _p(), rows, E, 8, cols, 0, _p(), None, None, None) == UNSUPPORTED
        assert L.hstu_expert_proj_e4m3(_p(), _p(), _p(), _p(), _p(), rows, E, 16, cols, 0, _p(), None,
                                       None) == UNSUPPORTED
        assert L.hstu_expert_proj_bwd(_p(), _p(), _p(), _p(), None, rows, E, cols, 8, _p(), None, None, None,
                                      0, None) == UNSUPPORTED
