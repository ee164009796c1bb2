"""GPU parity of the row operators (moe_quantize_rows, moe_combine and its
gradients) with the fp64 oracle, and runs of the separate operators together:
an MoE layer in 8 bits, and a training step of one.

Codes and scales are decided exactly, so they are compared for equality.  A
combine of k products in fp32 is within k 2^-24 sum|w y| of the exact sum, and
half a step of its output type; a dot product of n within 8 sqrt(n) 2^-23
sum|a b| (the probabilistic bound of n roundings of one fp32 step at most)."""
import numpy as np
import pytest
import torch

import oracle
import synth
from oracle import grouped as G
from tests import helpers as H

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module")
def m():
    return H.lib()



def tt(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def dev(a, dtype=None):
    t = torch.as_tensor(np.ascontiguousarray(a), device="cuda")
    return t if dtype is None else t.to(dtype)


# --------------------------------------------------------------- quantise --

def quantize(m, x):
    q = torch.full(tuple(x.shape), 99, dtype=torch.int8, device="cuda")
    s = torch.full((x.shape[0],), -7.0, device="cuda")
    m.moe_quantize_rows(x, q, s)
    return q.cpu().numpy().astype(np.int64), s.cpu().numpy()


def same_codes(m, x):
    q, s = quantize(m, x)
    rq, rs = G.quantize_rows(H.to_f64(x))
    assert np.array_equal(s, rs, equal_nan=True)
    assert np.array_equal(q, rq), (np.argwhere(q != rq)[:5], q[q != rq][:5], rq[q != rq][:5])


@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("rows, cols", [(1, 1), (1, 7), (3, 8), (5, 64), (2, 255), (4, 256), (3, 1000), (2, 2049),
                                        (1, 8192), (1, 8200), (2, 14336), (1, 100003), (700, 72)])
def test_codes(m, rows, cols, x):
    rng = np.random.default_rng(rows * 7 + cols)
    same_codes(m, dev((rng.normal(size=(rows, cols)) * 10.0 ** rng.integers(-3, 4, (rows, 1))).astype(np.float32), tt(x)))


def test_codes_at_halves(m):
    """Values on and one step beside the borders between codes, for scales that are not powers of two."""
    rng = np.random.default_rng(2)
    rows = []
    for _ in range(64):
        s = np.float32(rng.uniform(0.5, 2.0)) if rng.random() < 0.7 else np.float32(1.0)
        top = np.float32(np.float64(s) * 127)
        scale = np.float32(np.float64(top) / 127.0)
        mids = ((rng.integers(-127, 127, 40) + 0.5) * np.float64(scale)).astype(np.float32)
        rows.append(np.concatenate([[top], mids, np.nextafter(mids, np.float32(np.inf)),
                                    np.nextafter(mids, np.float32(-np.inf))]))
    same_codes(m, dev(np.array(rows, dtype=np.float32)))


def test_codes_of_unusual_rows(m):
    tiny, huge = 2.0 ** -149, 3.0e38
    rows = np.zeros((10, 9), dtype=np.float32)
    rows[1, 4] = tiny                        # its scale rounds to zero
    rows[2] = [100 * tiny, -64 * tiny, tiny, 0, 0, 0, 0, 0, 127 * tiny]
    rows[3, :2] = huge, -huge
    rows[4, 2] = np.nan
    rows[5, 3] = -np.inf
    rows[6] = -0.0
    rows[7] = 1.0
    rows[8] = [1e-30, 1, -1, 0.5, 0.003937008, -0.0039, 0.00393, 1e-3, 0.9961]
    rows[9] = np.array([191, -190, 64, 95, 63, 1, 2, 0, -95], dtype=np.float32) * tiny
    same_codes(m, dev(rows))
    for i in range(10):                      # a row's neighbours do not matter
        same_codes(m, dev(rows[i:i + 1]))


# ---------------------------------------------------------------- combine --

def combine_inputs(T, k, Hd, rows, y, out, seed=0, drop=0.2, distinct=True):
    rng = np.random.default_rng(seed)
    n = T * k
    inv = rng.permutation(max(rows, n))[:n] if distinct else rng.integers(0, max(rows, 1), n)
    inv = np.where(rng.random(n) < drop, rng.choice([-1, rows, 2147483647, -2147483648], n), inv)
    return (dev(rng.normal(size=(rows, Hd)).astype(np.float32), tt(y)), inv.astype(np.int32).reshape(T, k),
            rng.uniform(-1, 1, (T, k)).astype(np.float32), dev(rng.normal(size=(T, Hd)).astype(np.float32), tt(out)))


SIZES = [(1, 1, 1, 1), (1, 8, 2048, 8), (3, 2, 7, 9), (5, 3, 129, 20), (64, 6, 264, 400), (33, 1, 1000, 33),
         (7, 5, 1001, 40), (2, 256, 40, 600), (300, 2, 520, 1000), (4, 4, 8192, 16), (3, 2, 16, 0)]


@pytest.mark.parametrize("y, out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("T, k, Hd, rows", SIZES)
def test_combine(m, T, k, Hd, rows, y, out):
    for weighted in (True, False):
        yt, inv, w, _ = combine_inputs(T, k, Hd, rows, y, out, seed=T + Hd, distinct=False)
        got = torch.full((T, Hd), -7.0, dtype=tt(out), device="cuda")
        s = m.make_combine_shape(T, k, Hd, rows, y, out)
        m.moe_combine(s, yt, dev(inv), dev(w) if weighted else None, got)
        y64 = H.to_f64(yt)
        ref = G.combine(y64, inv, w if weighted else None)
        mag = G.combine(abs(y64), inv, abs(w) if weighted else None)
        bad = np.abs(H.to_f64(got) - ref) > HALF[out] * abs(ref) + k * 2.0 ** -24 * mag + 1e-40
        assert not bad.any(), np.argwhere(bad)[:4]


@pytest.mark.parametrize("y, out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("T, k, Hd, rows", SIZES)
def test_combine_backward(m, T, k, Hd, rows, y, out):
    yt, inv, w, dout = combine_inputs(T, k, Hd, rows, y, out, seed=T + Hd)
    s = m.make_combine_shape(T, k, Hd, rows, y, out)
    for weighted in (True, False):
        wt = dev(w) if weighted else None
        dy = torch.full((rows, Hd), -7.0, dtype=tt(y), device="cuda")
        dw = torch.full((T, k), -7.0, device="cuda")
        m.moe_combine_backward(s, dout, yt, dev(inv), wt, dy, dw)
        y64, g64 = H.to_f64(yt), H.to_f64(dout)
        rdy, rdw = G.combine_backward(g64, y64, inv, w if weighted else None)
        got = H.to_f64(dy)
        bad = ~np.isnan(rdy) & ~(np.abs(got - rdy) <= (HALF[y] + 2.0 ** -24) * abs(rdy) + 1e-40)
        assert not bad.any(), np.argwhere(bad)[:4]
        assert (got[np.isnan(rdy)] == -7.0).all()                  # rows that no assignment names
        mag = G.combine_backward(abs(g64), abs(y64), inv, None)[1]
        assert (np.abs(H.to_f64(dw) - rdw) <= 8 * np.sqrt(Hd) * 2.0 ** -23 * mag + 2.0 ** -24 * abs(rdw)).all()
        # each gradient by itself
        dy2, dw2 = torch.full_like(dy, -7.0), torch.full_like(dw, -7.0)
        m.moe_combine_backward(s, dout, None, dev(inv), wt, dy2, None)
        m.moe_combine_backward(s, dout, yt, dev(inv), wt, None, dw2)
        assert torch.equal(dy2, dy) and torch.equal(dw2, dw)


def test_combine_nan_and_infinity(m):
    """A dropped row's NaN does not reach the sum, a weight of 0 does not hide one."""
    y = torch.ones(4, 24, device="cuda")
    y[1], y[2, 3] = float("nan"), float("inf")
    inv = dev(np.array([[0, 3], [0, -1], [0, 1], [0, 2]], dtype=np.int32))
    w = torch.tensor([[1.0, 1.0], [1.0, float("nan")], [1.0, 0.0], [1.0, -1.0]], device="cuda")
    out = torch.empty(4, 24, device="cuda")
    m.moe_combine(m.make_combine_shape(4, 2, 24, 4, "f32", "f32"), y, inv, w, out)
    assert (out[0] == 2).all() and (out[1] == 1).all() and torch.isnan(out[2]).all()
    assert out[3, 3] == -float("inf") and (out[3, :3] == 0).all()


def test_combine_past_32_bit_offsets(m):
    """Rows of 2.2e9 elements, in both directions."""
    rows, Hd = 140000, 16000
    y = torch.empty(rows, Hd, dtype=torch.bfloat16, device="cuda").normal_()
    inv = dev(np.array([[rows - 1, 0], [rows - 2, 70000]], dtype=np.int32))
    w = torch.tensor([[0.5, 2.0], [1.0, -1.0]], device="cuda")
    out = torch.empty(2, Hd, device="cuda")
    s = m.make_combine_shape(2, 2, Hd, rows, "bf16", "f32")
    m.moe_combine(s, y, inv, w, out)
    ref = torch.stack([0.5 * y[rows - 1].double() + 2 * y[0].double(), y[rows - 2].double() - y[70000].double()])
    assert ((out.double() - ref).abs() <= 4 * 2.0 ** -24 * 20).all()
    last, dout = y[rows - 2].clone(), torch.randn(2, Hd, device="cuda")
    m.moe_combine_backward(s, dout, None, inv, w, y, None)
    assert torch.equal(y[rows - 1], (dout[0] * 0.5).bfloat16()) and torch.equal(y[rows - 2], dout[1].bfloat16())
    assert not torch.equal(y[rows - 2], last)


def test_row_operators_in_a_graph_and_on_a_stream(m):
    T, k, Hd, rows = 40, 3, 264, 130
    y, inv, w, dout = combine_inputs(T, k, Hd, rows, "bf16", "bf16")
    inv, w = dev(inv), dev(w)
    s = m.make_combine_shape(T, k, Hd, rows)
    out, dy, dw = torch.zeros_like(dout), torch.zeros_like(y), torch.zeros(T, k, device="cuda")
    q, sc = torch.zeros(rows, Hd, dtype=torch.int8, device="cuda"), torch.zeros(rows, device="cuda")

    def step():
        m.moe_combine(s, y, inv, w, out)
        m.moe_combine_backward(s, dout, y, inv, w, dy, dw)
        m.moe_quantize_rows(y, q, sc)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        y.normal_()
        dout.normal_()
        w.uniform_()
        for t in (out, dy, dw, q, sc):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out, dy, dw, q, sc)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (out, dy, dw, q, sc))), i


# ---------------------------------------------------------- runs together --

def route(m, wl, t):
    """moe_route's tables (torch, on the GPU) and their padded order's length."""
    s = H.shape_of(m, wl)
    tile_m, cap, n_tiles = m.moe_dispatch_dims(s)
    i32 = dict(dtype=torch.int32, device="cuda")
    n = wl.T * wl.k
    r = dict(topk_ids=torch.empty(n, **i32), topk_w=torch.empty(n, device="cuda"), counts=torch.empty(wl.E, **i32),
             offsets=torch.empty(wl.E + 1, **i32), sorted_ids=torch.empty(cap, **i32), inv=torch.empty(n, **i32))
    m.moe_route(s, t["x"], t["router_w"], t["router_b"], r, m.alloc_workspace(s, t["x"].device))
    return r, cap


@pytest.mark.parametrize("T, Hd, E, I, k", [(1, 64, 8, 96, 2), (37, 128, 6, 160, 3), (150, 256, 4, 320, 2)])
def test_layer_in_8_bits(m, T, Hd, E, I, k):
    """moe_route, then the three products of a SwiGLU layer on 8-bit codes and the combine, in moe_route's padded
    order, against the oracle's layer on the same codes."""
    wl = synth.WORKLOADS["tiny_f32"].replace(T=T, H=Hd, E=E, I=I, k=k, x_dtype="bf16", w_dtype="bf16", r_dtype="f32")
    inp = synth.make_inputs(wl, T)
    t = synth.to_torch(inp, torch.device("cuda"))
    r, cap = route(m, wl, t)
    codes = {}
    for name in ("w_gate", "w_up", "w_down"):
        w = t[name].reshape(-1, t[name].shape[-1])
        q, sc = torch.empty(w.shape, dtype=torch.int8, device="cuda"), torch.empty(w.shape[0], device="cuda")
        m.moe_quantize_rows(w, q, sc)
        codes[name] = (q, sc)
    xq, xs = torch.empty(T, Hd, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    m.moe_quantize_rows(t["x"], xq, xs)
    up = m.make_grouped_shape(cap, I, Hd, E, x_rows=T, row_div=k, x_dtype="i8", out_dtype="f32")
    g, u = torch.zeros(cap, I, device="cuda"), torch.zeros(cap, I, device="cuda")
    for out, name in ((g, "w_gate"), (u, "w_up")):
        m.moe_grouped_matmul_i8(up, xq, xs, r["sorted_ids"], r["offsets"], r["counts"], *codes[name], out,
                                m.alloc_grouped_workspace(up))
    h = torch.nn.functional.silu(g) * u
    hq, hs = torch.empty(cap, I, dtype=torch.int8, device="cuda"), torch.empty(cap, device="cuda")
    m.moe_quantize_rows(h, hq, hs)
    down = m.make_grouped_shape(cap, Hd, I, E, x_dtype="i8", out_dtype="f32")
    y = torch.empty(cap, Hd, device="cuda")
    m.moe_grouped_matmul_i8(down, hq, hs, None, r["offsets"], r["counts"], *codes["w_down"], y,
                            m.alloc_grouped_workspace(down))
    out = torch.empty(T, Hd, device="cuda")
    m.moe_combine(m.make_combine_shape(T, k, Hd, cap, "f32", "f32"), y, r["inv"], r["topk_w"], out)

    # the oracle on the values that the codes stand for; the hidden codes are the GPU's own
    value = lambda q, sc: q.double().cpu().numpy() * sc.double().cpu().numpy()[:, None]
    W = {n: value(*codes[n]).reshape(E, -1, codes[n][0].shape[1]) for n in codes}
    x64, ids = value(xq, xs), r["topk_ids"].cpu().numpy().reshape(T, k)
    inv, tw = r["inv"].cpu().numpy().reshape(T, k), r["topk_w"].double().cpu().numpy().reshape(T, k)
    h64, hv, ref = h.double().cpu().numpy(), value(hq, hs), np.zeros((T, Hd))
    for i in range(T):
        for j in range(k):
            e, p = ids[i, j], inv[i, j]
            a, b = W["w_gate"][e] @ x64[i], W["w_up"][e] @ x64[i]
            want = a / (1 + np.exp(-a)) * b
            # g and u carry three fp32 roundings each, the activation and the product a few more
            assert (abs(h64[p] - want) <= 24 * 2.0 ** -24 * (abs(a) + 1) * abs(b) + 1e-12).all()
            assert (abs(hv[p] - h64[p]) <= 0.5000001 * hs[p].item()).all()
            ref[i] += tw[i, j] * (W["w_down"][e] @ hv[p])
    assert H.relerr(out.double().cpu().numpy(), ref) < 1e-6 * k


def test_training_step(m):
    """Forward and backward of a gathered two-matrix layer (y = combine(W2 tanh(W1 x))) with moe_route's tables:
    every gradient against the 64-bit formula, and the loss's own differences."""
    T, Hd, E, I, k = 23, 64, 5, 96, 2
    wl = synth.WORKLOADS["tiny_f32"].replace(T=T, H=Hd, E=E, I=I, k=k)
    t = synth.to_torch(synth.make_inputs(wl, 3), torch.device("cuda"))
    r, cap = route(m, wl, t)
    w1, w2, x = t["w_gate"] * 4, t["w_down"] * 4, t["x"]
    up = m.make_grouped_shape(cap, I, Hd, E, x_rows=T, row_div=k, x_dtype="f32", out_dtype="f32")
    down = m.make_grouped_shape(cap, Hd, I, E, x_dtype="f32", out_dtype="f32")
    cs = m.make_combine_shape(T, k, Hd, cap, "f32", "f32")
    z = lambda *s: torch.zeros(*s, device="cuda")
    tab = (r["offsets"], r["counts"])
    a, y, out = z(cap, I), z(cap, Hd), z(T, Hd)
    m.moe_grouped_matmul(up, x, r["sorted_ids"], *tab, w1, a, m.alloc_grouped_workspace(up))
    h = torch.tanh(a)
    m.moe_grouped_matmul(down, h, None, *tab, w2, y, m.alloc_grouped_workspace(down))
    m.moe_combine(cs, y, r["inv"], r["topk_w"], out)
    dout = torch.randn(T, Hd, device="cuda")
    dy, dtw, dh, dw2, dxs, dw1, dx = z(cap, Hd), z(T, k), z(cap, I), z(E, Hd, I), z(cap, Hd), z(E, I, Hd), z(T, Hd)
    m.moe_combine_backward(cs, dout, y, r["inv"], r["topk_w"], dy, dtw)
    m.moe_grouped_matmul_backward(down, dy, h, None, *tab, w2, dh, dw2, m.alloc_grouped_workspace(down))
    da = dh * (1 - h * h)
    m.moe_grouped_matmul_backward(up, da, x, r["sorted_ids"], *tab, w1, dxs, dw1, m.alloc_grouped_workspace(up))
    m.moe_combine(cs, dxs, r["inv"], None, dx)

    ids = r["topk_ids"].cpu().long().view(T, k)
    leaves = [v.double().cpu().requires_grad_() for v in (x, w1, w2, r["topk_w"].view(T, k))]

    def loss(x, w1, w2, tw):
        o = torch.zeros(T, Hd, dtype=torch.float64)
        for j in range(k):
            hid = torch.tanh((w1[ids[:, j]] * x[:, None, :]).sum(2))
            o = o + tw[:, j, None] * (w2[ids[:, j]] * hid[:, None, :]).sum(2)
        return o, (o * dout.double().cpu()).sum()

    o, L = loss(*leaves)
    L.backward()
    assert H.relerr(out.double().cpu().numpy(), o.detach().numpy()) < 1e-5
    for got, leaf in zip((dx, dw1, dw2, dtw), leaves):
        assert H.relerr(got.double().cpu().numpy(), leaf.grad.numpy()) < 1e-5
    rng = np.random.default_rng(0)
    plain = [v.detach() for v in leaves]
    for got, i in ((dx, 0), (dw1, 1), (dw2, 2), (dtw, 3)):
        for _ in range(3):
            at = tuple(int(rng.integers(n)) for n in plain[i].shape)
            d = torch.zeros_like(plain[i])
            d[at] = 1e-4
            up_, dn = list(plain), list(plain)
            up_[i], dn[i] = plain[i] + d, plain[i] - d
            want = float(loss(*up_)[1] - loss(*dn)[1]) / 2e-4
            assert abs(float(got[at]) - want) <= 1e-5 * float(got.abs().max()) + 1e-6
