"""CPU checks of the separate operators (grouped expert products, 8-bit row
codes, combine): hand-worked pins of their fp64 oracle, its gradients against
differences, and the refusals of the C ABI and of the binding, all before
anything is launched."""
import ctypes

import numpy as np
import pytest

from oracle import grouped as G
from tests import helpers as H


@pytest.fixture(scope="module")
def m():
    return H.lib()


# ---------------------------------------------------------------- oracle --

def test_segments_are_cut_to_the_rows():
    assert G.segments([0, 3, 3, 9], None, 7, 3) == [(0, 3), (3, 3), (3, 7)]
    assert G.segments([0, 4, 8], [2, 0, -5], 10, 3) == [(0, 2), (4, 4), (8, 8)]
    assert G.segments([-2, 6], [5, 100], 10, 2) == [(0, 3), (6, 10)]


def test_product_by_hand():
    w = np.array([[[1.0, 2.0]], [[3.0, -1.0]]])                  # two experts, N = 1, K = 2
    x = np.array([[1.0, 1.0], [2.0, 0.0]])
    xs = G.lookup(x, np.array([3, 0, -1, 9]), 2, 4)              # rows 1, 0, zeros, past the end
    assert xs.tolist() == [[2, 0], [1, 1], [0, 0], [0, 0]]
    y = G.grouped_matmul(xs, [(0, 1), (1, 3)], w)
    assert y[:3, 0].tolist() == [2.0, 2.0, 0.0] and np.isnan(y[3, 0])


def test_codes_by_hand():
    q, s = G.quantize_rows(np.array([[127.0, -63.5, 0.5, 1.5, 2.5], [0, 0, 0, 0, 0], [1, np.inf, 0, 0, 0]]))
    assert s[0] == 1.0 and q[0].tolist() == [127, -64, 0, 2, 2]   # halves go to the even code
    assert s[1] == 0.0 and not q[1].any()
    assert np.isnan(s[2]) and not q[2].any()


def test_combine_by_hand():
    y = np.array([[1.0], [10.0], [100.0]])
    inv = np.array([[2, 0], [-1, 3], [1, -1]])
    w = np.array([[0.5, 2.0], [1.0, 1.0], [0.25, 1.0]])
    assert G.combine(y, inv, w)[:, 0].tolist() == [52.0, 0.0, 2.5]
    assert G.combine(y, inv, None)[:, 0].tolist() == [101.0, 0.0, 10.0]
    dy, dw = G.combine_backward(np.array([[3.0], [5.0], [7.0]]), y, inv, w)
    assert dy[:, 0].tolist() == [6.0, 1.75, 1.5] and dw.tolist() == [[300.0, 3.0], [0.0, 0.0], [70.0, 0.0]]


def test_gradients_against_differences():
    rng = np.random.default_rng(0)
    rows, N, K, E = 7, 3, 4, 3
    segs = [(0, 2), (2, 2), (3, 7)]
    xs, w, dy = rng.normal(size=(rows, K)), rng.normal(size=(E, N, K)), rng.normal(size=(rows, N))
    loss = lambda xs, w: np.nansum(G.grouped_matmul(xs, segs, w) * dy)
    dx, dw = G.grouped_matmul_backward(dy, xs, segs, w)
    h = 1e-3                                                     # the loss is linear in each: no truncation error
    for idx in np.ndindex(*xs.shape):
        d = np.zeros_like(xs)
        d[idx] = h
        want = (loss(xs + d, w) - loss(xs - d, w)) / (2 * h)
        assert abs((0.0 if np.isnan(dx[idx]) else dx[idx]) - want) < 1e-9
    for idx in np.ndindex(*w.shape):
        d = np.zeros_like(w)
        d[idx] = h
        assert abs(dw[idx] - (loss(xs, w + d) - loss(xs, w - d)) / (2 * h)) < 1e-9


# -------------------------------------------------------------- refusals --

GOOD = dict(rows=16, N=8, K=8, E=2, x_rows=16, row_div=1, x_dtype=1, out_dtype=1)


@pytest.mark.parametrize("kw, code", [
    (dict(rows=-1), "MOE_ERR_SHAPE"), (dict(rows=33554433), "MOE_ERR_SHAPE"), (dict(x_rows=-1), "MOE_ERR_SHAPE"),
    (dict(N=0), "MOE_ERR_SHAPE"), (dict(K=0), "MOE_ERR_SHAPE"), (dict(N=1048577), "MOE_ERR_SHAPE"),
    (dict(K=1048577), "MOE_ERR_SHAPE"), (dict(E=0), "MOE_ERR_SHAPE"), (dict(E=257), "MOE_ERR_SHAPE"),
    (dict(row_div=0), "MOE_ERR_SHAPE"), (dict(row_div=257), "MOE_ERR_SHAPE"),
    (dict(x_dtype=2), "MOE_ERR_DTYPE"), (dict(x_dtype=6), "MOE_ERR_DTYPE"), (dict(out_dtype=5), "MOE_ERR_DTYPE"),
    (dict(x_dtype=0), "MOE_ERR_DTYPE"),                            # fp32 inputs round to no narrower output
    (dict(x_dtype=5, K=131072), "MOE_ERR_SHAPE"),                  # a sum of 8-bit products could pass 31 bits
])
def test_grouped_shape_is_checked(m, kw, code):
    s = m.moe_grouped_shape_t(*[{**GOOD, **kw}[n] for n, _ in m.moe_grouped_shape_t._fields_])
    n = ctypes.c_size_t(0)
    assert m.load_library().moe_grouped_workspace_size(ctypes.byref(s), ctypes.byref(n)) == getattr(m, code)


def _shape(m, **kw):
    return m.moe_grouped_shape_t(*[{**GOOD, **kw}[n] for n, _ in m.moe_grouped_shape_t._fields_])


P = 4096          # an aligned address that is never read: every call below is refused first
BIG = 1 << 40


def test_forward_arguments_are_checked(m):
    s = _shape(m)
    call = lambda s=s, x=P, ids=None, off=P, cnt=None, w=P, y=P, ws=P, nb=BIG: m.moe_grouped_matmul(
        s, x, ids, off, cnt, w, y, ws, ws_bytes=nb, stream=0, check=False)
    assert call(x=None) == call(off=None) == call(w=None) == call(y=None) == m.MOE_ERR_NULL
    for name in ("x", "ids", "off", "cnt", "w", "y", "ws"):
        assert call(**{name: P + 4}) == m.MOE_ERR_ALIGN
    assert call(s=_shape(m, x_dtype=5)) == m.MOE_ERR_DTYPE         # 8-bit codes have a call of their own
    assert call(s=_shape(m, x_rows=15)) == m.MOE_ERR_SHAPE         # without row_ids row r is row r
    assert call(s=_shape(m, row_div=2)) == m.MOE_ERR_SHAPE
    assert call(s=_shape(m, rows=0, x_rows=0), x=None, off=None, w=None, y=None, ws=None, nb=0) == m.MOE_OK
    # every size whose calls need a workspace refuses one that is a byte short
    for kw in (dict(), dict(rows=1, x_rows=1, N=512, K=16384), dict(rows=512, x_rows=512, N=256, K=8192)):
        big = _shape(m, **kw)
        need = m.moe_grouped_workspace_size(big)
        if need:
            assert call(s=big, nb=need - 1) == m.MOE_ERR_WORKSPACE and call(s=big, ws=None) == m.MOE_ERR_NULL


def test_backward_arguments_are_checked(m):
    s = _shape(m)
    call = lambda s=s, dy=P, x=P, ids=None, off=P, cnt=None, w=P, dx=P, dw=P, ws=P, nb=BIG: \
        m.moe_grouped_matmul_backward(s, dy, x, ids, off, cnt, w, dx, dw, ws, ws_bytes=nb, stream=0, check=False)
    assert call(dx=None, dw=None) == m.MOE_ERR_NULL
    assert call(dy=None) == call(off=None) == call(w=None) == call(x=None) == m.MOE_ERR_NULL
    assert call(w=None, dx=None, x=None) == call(x=None, dw=None, w=None) == m.MOE_ERR_NULL
    for name in ("dy", "x", "ids", "off", "cnt", "w", "dx", "dw", "ws"):
        assert call(**{name: P + 8}) == m.MOE_ERR_ALIGN
    assert call(s=_shape(m, x_dtype=5)) == m.MOE_ERR_DTYPE
    assert call(s=_shape(m, x_rows=15)) == m.MOE_ERR_SHAPE
    assert call(s=_shape(m, rows=0, x_rows=0), dy=None, dw=None, x=None, off=None, w=None) == m.MOE_OK


def test_i8_arguments_are_checked(m):
    s = _shape(m, x_dtype=5)
    call = lambda s=s, x=P, xs=P, ids=None, off=P, cnt=None, w=P, wsc=P, y=P, ws=P, nb=BIG: m.moe_grouped_matmul_i8(
        s, x, xs, ids, off, cnt, w, wsc, y, ws, ws_bytes=nb, stream=0, check=False)
    for name in ("x", "xs", "off", "w", "wsc", "y"):
        assert call(**{name: None}) == m.MOE_ERR_NULL
        assert call(**{name: P + 1}) == m.MOE_ERR_ALIGN
    assert call(s=_shape(m)) == m.MOE_ERR_DTYPE
    assert call(s=_shape(m, x_dtype=5, x_rows=3)) == m.MOE_ERR_SHAPE


def test_quantize_arguments_are_checked(m):
    f = m.load_library().moe_quantize_rows
    assert f(-1, 8, 1, P, P, P, None) == f(33554433, 8, 1, P, P, P, None) == m.MOE_ERR_SHAPE
    assert f(4, 0, 1, P, P, P, None) == f(4, 1048577, 1, P, P, P, None) == m.MOE_ERR_SHAPE
    assert f(4, 8, 5, P, P, P, None) == f(4, 8, 2, P, P, P, None) == m.MOE_ERR_DTYPE
    assert f(4, 8, 1, None, P, P, None) == f(4, 8, 1, P, None, P, None) == f(4, 8, 1, P, P, None, None) == m.MOE_ERR_NULL
    assert f(4, 8, 1, P + 2, P, P, None) == f(4, 8, 1, P, P + 1, P, None) == f(4, 8, 1, P, P, P + 4, None) == \
        m.MOE_ERR_ALIGN
    assert f(0, 8, 1, None, None, None, None) == m.MOE_OK


@pytest.mark.parametrize("kw, code", [
    (dict(T=-1), "MOE_ERR_SHAPE"), (dict(T=1048577), "MOE_ERR_SHAPE"), (dict(top_k=0), "MOE_ERR_SHAPE"),
    (dict(top_k=257), "MOE_ERR_SHAPE"), (dict(T=1048576, top_k=17), "MOE_ERR_SHAPE"), (dict(H=0), "MOE_ERR_SHAPE"),
    (dict(H=1048577), "MOE_ERR_SHAPE"), (dict(rows=-1), "MOE_ERR_SHAPE"), (dict(rows=33554433), "MOE_ERR_SHAPE"),
    (dict(y_dtype=5), "MOE_ERR_DTYPE"), (dict(out_dtype=2), "MOE_ERR_DTYPE"),
])
def test_combine_shape_is_checked(m, kw, code):
    base = dict(T=4, top_k=2, H=8, rows=8, y_dtype=1, out_dtype=1)
    s = m.moe_combine_shape_t(*[{**base, **kw}[n] for n, _ in m.moe_combine_shape_t._fields_])
    assert m.moe_combine(s, P, P, P, P, stream=0, check=False) == getattr(m, code)
    assert m.moe_combine_backward(s, P, P, P, P, P, P, stream=0, check=False) == getattr(m, code)


def test_combine_arguments_are_checked(m):
    s = m.make_combine_shape(4, 2, 8, 8)
    call = lambda y=P, inv=P, w=P, out=P: m.moe_combine(s, y, inv, w, out, stream=0, check=False)
    assert call(y=None) == call(inv=None) == call(out=None) == m.MOE_ERR_NULL
    back = lambda dout=P, y=P, inv=P, w=P, dy=P, dw=P: m.moe_combine_backward(s, dout, y, inv, w, dy, dw, stream=0,
                                                                             check=False)
    assert back(dy=None, dw=None) == back(dout=None) == back(y=None) == back(inv=None) == m.MOE_ERR_NULL
    for name in ("y", "inv", "w"):
        assert call(**{name: P + 4}) == back(**{name: P + 4}) == m.MOE_ERR_ALIGN
    assert call(out=P + 4) == back(dy=P + 4) == back(dw=P + 4) == back(dout=P + 2) == m.MOE_ERR_ALIGN
    assert m.moe_combine(m.make_combine_shape(0, 2, 8, 8), None, None, None, None, stream=0, check=False) == m.MOE_OK


def test_binding_checks_tensors(m):
    import torch
    s = m.make_grouped_shape(4, 8, 8, 1)
    x, w, y = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(1, 8, 8, dtype=torch.bfloat16), None
    off = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="not on a GPU"):
        m.moe_grouped_matmul(s, x, None, off, None, w, P, P, ws_bytes=0, stream=0)
    with pytest.raises(ValueError, match="not contiguous"):
        m.moe_grouped_matmul(s, torch.zeros(8, 4, dtype=torch.bfloat16).t(), None, P, None, P, P, P, ws_bytes=0,
                             stream=0)
    with pytest.raises(ValueError, match="has type"):
        m.moe_grouped_matmul(s, x.float(), None, P, None, P, P, P, ws_bytes=0, stream=0)
    with pytest.raises(ValueError, match="elements"):
        m.moe_grouped_matmul(s, x[:3], None, P, None, P, P, P, ws_bytes=0, stream=0)
    with pytest.raises(ValueError, match="elements"):             # without counts the offsets end with the total
        m.moe_grouped_matmul(s, P, None, off[:1], None, P, P, P, ws_bytes=0, stream=0)
    with pytest.raises(ValueError):
        m.moe_quantize_rows(torch.zeros(4, dtype=torch.float32), P, P, stream=0)
