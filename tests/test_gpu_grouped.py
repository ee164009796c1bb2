"""GPU parity of the grouped expert products (moe_grouped_matmul and its
gradients, moe_grouped_matmul_i8) with the fp64 oracle.

Tolerances, element by element: half a step of the output type relative to the
value, plus the error of an fp32 sum of n products, 8 sqrt(n) 2^-23 sum|a b|
(the probabilistic bound of a sum of n roundings of at most one fp32 step each
with a factor of 8, n the reduction's length).  An 8-bit sum is exact, and
three fp32 roundings (the conversion and two scales) of 2^-24 follow."""
import numpy as np
import pytest
import torch

from oracle import grouped as G
from tests import helpers as H

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module")
def m():
    return H.lib()



def dev(a, dtype=None):
    t = torch.as_tensor(np.ascontiguousarray(a), device="cuda")
    return t if dtype is None else t.to(dtype)


TYPES = {"bf16": "bfloat16", "f32": "float32"}


def tt(name):
    return getattr(torch, TYPES[name])


def close(got, ref, mag, n, out):
    """got within the tolerance of ref wherever ref is a number; mag = sum |a b|."""
    ok = ~np.isnan(ref)
    tol = HALF[out] * np.abs(ref) + 8 * np.sqrt(n) * 2.0 ** -23 * mag + 1e-37
    bad = ok & ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], ref[bad][:4], tol[bad][:4])


SENTINEL = -777.0     # what outputs hold before a call


class Case:
    """Inputs of one product: float arrays hold values that their type represents exactly."""

    def __init__(self, counts, N, K, x="bf16", out="bf16", pad=1, use_counts=True, ids=None, row_div=1, x_rows=None,
                 rows=None, extra_rows=0, seed=0, ints=False):
        rng = np.random.default_rng(seed)
        counts = np.asarray(counts, dtype=np.int64)
        self.E, self.N, self.K, self.x_dt, self.out_dt = len(counts), N, K, x, out
        off = np.zeros(self.E + 1, dtype=np.int64)
        off[1:] = np.cumsum((counts + pad - 1) // pad * pad)
        self.rows = int(off[-1]) + extra_rows if rows is None else rows
        self.row_div = row_div
        self.x_rows = self.rows if ids is None else x_rows
        self.ids = None if ids is None else np.asarray(ids(rng, self.rows), dtype=np.int32)
        draw = (lambda *s: rng.integers(-3, 4, s).astype(np.float32)) if ints else \
            (lambda *s: rng.normal(size=s).astype(np.float32))
        self.x, self.w = dev(draw(self.x_rows, K), tt(x)), dev(draw(self.E, N, K), tt(x))
        self.dy = dev(draw(self.rows, N), tt(x))
        self.offsets, self.counts = dev(off.astype(np.int32)), dev(counts.astype(np.int32)) if use_counts else None
        self.segs = G.segments(off, counts if use_counts else None, self.rows, self.E)
        self.ids_t = None if self.ids is None else dev(self.ids)

    def shape(self, m, x=None):
        return m.make_grouped_shape(self.rows, self.N, self.K, self.E, self.x_rows, self.row_div, x or self.x_dt,
                                    self.out_dt)

    def ws(self, m, shape):
        w = m.alloc_grouped_workspace(shape)
        w.fill_(0xA5)                                   # nothing is expected of its contents
        return w

    def forward(self, m, stream=None):
        s = self.shape(m)
        y = torch.full((self.rows, self.N), SENTINEL, dtype=tt(self.out_dt), device="cuda")
        m.moe_grouped_matmul(s, self.x, self.ids_t, self.offsets, self.counts, self.w, y, self.ws(m, s), stream=stream)
        return y

    def backward(self, m, dx=True, dw=True):
        s = self.shape(m)
        gx = torch.full((self.rows, self.K), SENTINEL, dtype=tt(self.x_dt), device="cuda") if dx else None
        gw = torch.full((self.E, self.N, self.K), SENTINEL, dtype=tt(self.out_dt), device="cuda") if dw else None
        m.moe_grouped_matmul_backward(s, self.dy, self.x, self.ids_t, self.offsets, self.counts, self.w, gx, gw,
                                      self.ws(m, s))
        return gx, gw

    def check(self, m, backward=True):
        xs, w, dy = G.lookup(H.to_f64(self.x), self.ids, self.row_div, self.rows), H.to_f64(self.w), H.to_f64(self.dy)
        self.check_part(G.grouped_matmul(xs, self.segs, w), G.grouped_matmul(abs(xs), self.segs, abs(w)),
                        H.to_f64(self.forward(m)), self.K, self.out_dt)
        if backward:
            gx, gw = self.backward(m)
            rx, rw = G.grouped_matmul_backward(dy, xs, self.segs, w)
            ax, aw = G.grouped_matmul_backward(abs(dy), abs(xs), self.segs, abs(w))
            self.check_part(rx, ax, H.to_f64(gx), self.N, self.x_dt)
            longest = max([1] + [b - a for a, b in self.segs])
            close(H.to_f64(gw), rw, aw, longest, self.out_dt)

    def check_part(self, ref, mag, got, n, out):
        close(got, ref, mag, n, out)
        untouched = np.isnan(ref).all(axis=1)
        assert (got[untouched] == float(torch.tensor(SENTINEL).to(tt(out)))).all()


lookup = lambda n_ids: (lambda rng, rows: rng.integers(0, n_ids, rows))

COUNTS = [
    [1], [5], [128], [129], [300], [0], [0, 0, 3], [1, 0, 127, 128, 0, 130], [17, 2, 0, 64, 65, 255, 256, 257],
]


@pytest.mark.parametrize("x, out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("counts", COUNTS)
def test_segments(m, counts, x, out):
    Case(counts, 96, 64, x, out, extra_rows=3).check(m)


@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("N, K", [(1, 1), (2, 3), (7, 31), (33, 65), (129, 127), (130, 8), (8, 130), (255, 257),
                                  (256, 256), (257, 1000), (1001, 72), (512, 2048), (64, 4096)])
def test_sizes(m, N, K, x):
    Case([3, 0, 140], N, K, x, x, seed=N * 31 + K).check(m)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("counts", [[1, 0, 63, 64], [65, 128, 129], [255, 256, 257, 0, 5], [600]])
@pytest.mark.parametrize("N, K", [(1032, 1096), (1288, 1024), (1100, 2056)])
def test_long_reductions(m, N, K, counts, out):
    """Both products of at least 16 stages: large tiles of every height, whole and cut along the reduction, whose
    ends lie inside a stage and inside a tile; rows behind and between the segments stay."""
    Case(counts, N, K, "bf16", out, pad=3, extra_rows=9, seed=N + len(counts)).check(m)
    ids = lambda rng, rows: rng.integers(-3, 2 * 70 + 9, rows)
    Case(counts, N, K, "bf16", out, pad=2, ids=ids, row_div=2, x_rows=70, seed=N).check(m)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("lookup_rows", [False, True])
@pytest.mark.parametrize("N, K", [(264, 520), (512, 256), (40, 1288)])
def test_weight_gradients_of_many_tiles(m, N, K, lookup_rows, out):
    """Enough tiles of dw for the resident work-groups: segments of no row, of a part of a stage, of whole stages."""
    counts = [0, 1, 63, 64, 65, 127, 128, 129, 190, 200, 3] * 6
    kw = dict(ids=lambda rng, rows: rng.integers(-9, 3 * 500 + 40, rows), row_div=3, x_rows=500) if lookup_rows else {}
    c = Case(counts, N, K, "bf16", out, pad=4, extra_rows=5, seed=N, **kw)
    xs, dy = G.lookup(H.to_f64(c.x), c.ids, c.row_div, c.rows), H.to_f64(c.dy)
    w = np.zeros((c.E, N, K))
    gw = H.to_f64(c.backward(m, dx=False)[1])
    rw, aw = (G.grouped_matmul_backward(a, b, c.segs, w)[1] for a, b in ((dy, xs), (abs(dy), abs(xs))))
    close(gw, rw, aw, 200, out)
    assert (gw[0] == 0).all()


@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_few_tiles_are_cut(m, x):
    """Small outputs of long reductions, aligned and not: the parts add up, dw of short segments among them."""
    for N, K, counts in ((3, 5001, [2, 0, 40]), (5001, 3, [70, 1]), (16, 24, [3000, 0, 700, 5]), (17, 23, [2500, 9]),
                         (2000, 40, [33, 35]), (64, 4104, [200, 3])):
        Case(counts, N, K, x, x, pad=2, extra_rows=3, seed=K).check(m)


@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_padded_order_and_lookup(m, x):
    """moe_route's padded order: sentinel ids in the padding, rows looked up twice, never or outside x."""
    ids = lambda rng, rows: rng.integers(-4, 3 * 50 + 30, rows)      # tokens 0 .. 49 of 3 each; some outside
    Case([5, 0, 130, 128], 72, 88, x, x, pad=128, ids=ids, row_div=3, x_rows=50).check(m)
    Case([5, 0, 130, 128], 71, 89, x, x, pad=128, ids=ids, row_div=3, x_rows=50).check(m)


def test_offsets_without_counts(m):
    Case([4, 0, 9, 200], 40, 48, use_counts=False).check(m)


def test_many_experts(m):
    rng = np.random.default_rng(5)
    Case(rng.integers(0, 9, 256), 48, 40, seed=5).check(m)
    Case(rng.integers(0, 3, 256) * rng.integers(0, 130, 256), 16, 24, seed=6).check(m)


def test_tables_that_lead_outside_are_cut(m):
    """Offsets and counts past the rows, negative ones, and ids at the ends of 32 bits touch no other row."""
    c = Case([4, 4, 4], 24, 40, extra_rows=0)
    for off, cnt in [([-3, 4, 11], [5, 5, 2147483647]), ([0, 2147483647, -2147483648], [12, 5, 5]),
                     ([4, 0, 8], [4, 4, -1])]:
        c.offsets, c.counts = dev(np.array(off + [0], dtype=np.int32)), dev(np.array(cnt, dtype=np.int32))
        c.segs = G.segments(off + [0], cnt, c.rows, c.E)
        c.check(m)
    ids = np.array([2147483647, -2147483648, -1, 0, 5, 11, 12, 3, 3, 3, 1, 2], dtype=np.int32)
    d = Case([4, 4, 4], 24, 40, ids=lambda rng, rows: ids, row_div=1, x_rows=12)
    d.check(m)


@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_whole_numbers_come_out_exactly(m, x):
    """Products of small whole numbers are exact in fp32 whatever their order: any wrong index shows."""
    c = Case([130, 0, 3, 257], 136, 264, x, "f32", ints=True, ids=lookup(77 * 2), row_div=2, x_rows=77)
    xs, w, dy = G.lookup(H.to_f64(c.x), c.ids, 2, c.rows), H.to_f64(c.w), H.to_f64(c.dy)
    assert (H.to_f64(c.forward(m)) == G.grouped_matmul(xs, c.segs, w)).all()
    rx, rw = G.grouped_matmul_backward(dy, xs, c.segs, w)
    gx, gw = c.backward(m)
    assert (H.to_f64(gw) == rw).all()
    if x == "f32":
        assert (H.to_f64(gx) == rx).all()


def test_nan_and_infinity_stay_in_their_rows(m):
    """NaN in padding rows, in rows of x that nobody looks up and in experts without rows reach no output; an
    infinity reaches its own row only."""
    for K, N in ((64, 64), (67, 61)):
        c = Case([5, 0, 130], N, K, "bf16", "f32", pad=128, ids=lookup(40), row_div=1, x_rows=60)
        c.x[40:] = float("nan")
        c.w[1] = float("nan")
        used = np.zeros(c.rows, dtype=bool)
        for a, b in c.segs:
            used[a:b] = True
        c.ids[~used] = 50
        c.ids_t = dev(c.ids)
        c.dy[torch.as_tensor(~used, device="cuda")] = float("nan")
        y = c.forward(m)
        gx, gw = c.backward(m)
        u = torch.as_tensor(used, device="cuda")
        assert torch.isfinite(y[u]).all() and torch.isfinite(gx[u].float()).all() and torch.isfinite(gw).all()
        c.x[int(c.ids[0])] = float("inf")
        y2 = c.forward(m)
        same = torch.as_tensor(c.ids != c.ids[0], device="cuda") & u
        assert torch.equal(y2[same], y[same]) and not torch.isfinite(y2[0]).any()


def test_one_gradient_at_a_time(m):
    c = Case([7, 140], 72, 40)
    gx, gw = c.backward(m)
    assert torch.equal(c.backward(m, dw=False)[0], gx) and torch.equal(c.backward(m, dx=False)[1], gw)
    s = c.shape(m)
    only = torch.empty_like(gx)
    m.moe_grouped_matmul_backward(s, c.dy, None, None, c.offsets, c.counts, c.w, only, None, c.ws(m, s))
    assert torch.equal(only[:147], gx[:147])
    only = torch.empty_like(gw)
    m.moe_grouped_matmul_backward(s, c.dy, c.x, None, c.offsets, c.counts, None, None, only, c.ws(m, s))
    assert torch.equal(only, gw)


def test_no_rows_at_all(m):
    c = Case([0, 0], 40, 24)
    assert c.rows == 0
    gw = c.backward(m)[1]
    assert (gw == 0).all()
    c.forward(m)


@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_gradients_against_differences(m, x):
    """The loss sum(y * dy) is linear in x and in w: its central difference in 64 bits is the gradient."""
    c = Case([6, 0, 9], 12, 20, x, "f32", ids=lookup(8), row_div=1, x_rows=8)
    x64, w, dy = H.to_f64(c.x), H.to_f64(c.w), H.to_f64(c.dy)
    loss = lambda x64, w: np.nansum(G.grouped_matmul(G.lookup(x64, c.ids, 1, c.rows), c.segs, w) * dy)
    gx, gw = (H.to_f64(t) for t in c.backward(m))
    xs = G.lookup(x64, c.ids, 1, c.rows)
    ax, aw = G.grouped_matmul_backward(abs(dy), abs(xs), c.segs, abs(w))
    # the gradient of a looked-up row is the sum over the sorted rows that read it
    gxt, tol = np.zeros_like(x64), np.zeros_like(x64)
    for a, b in c.segs:
        for r in range(a, b):
            gxt[c.ids[r]] += gx[r]
            tol[c.ids[r]] += (HALF[x] + 8 * np.sqrt(12) * 2.0 ** -23) * ax[r]
    rng = np.random.default_rng(1)
    for _ in range(20):
        i = (rng.integers(8), rng.integers(20))
        d = np.zeros_like(x64)
        d[i] = 0.5
        assert abs(gxt[i] - (loss(x64 + d, w) - loss(x64 - d, w))) <= tol[i] + 1e-11
        j = (rng.choice([0, 2]), rng.integers(12), rng.integers(20))
        d = np.zeros_like(w)
        d[j] = 0.5
        want = loss(x64, w + d) - loss(x64, w - d)
        assert abs(gw[j] - want) <= (HALF["f32"] + 8 * 3 * 2.0 ** -23) * aw[j] + 1e-11


# ------------------------------------------------------------------- 8-bit --

def i8_case(m, counts, N, K, out="bf16", seed=0, **kw):
    c = Case(counts, N, K, "bf16", out, seed=seed, **kw)
    rng = np.random.default_rng(seed + 1)
    q = rng.integers(-128, 128, (c.x_rows, K)).astype(np.int8)
    wq = rng.integers(-128, 128, (c.E, N, K)).astype(np.int8)
    xs = rng.uniform(0.001, 0.1, c.x_rows).astype(np.float32)
    ws = rng.uniform(-0.01, 0.01, (c.E, N)).astype(np.float32)
    s = c.shape(m, "i8")
    y = torch.full((c.rows, N), SENTINEL, dtype=tt(out), device="cuda")
    m.moe_grouped_matmul_i8(s, dev(q), dev(xs), c.ids_t, c.offsets, c.counts, dev(wq), dev(ws), y, c.ws(m, s))
    ref = G.grouped_matmul_i8(q, xs, c.ids, c.row_div, c.segs, wq, ws, c.rows)
    got = H.to_f64(y)
    ok = ~np.isnan(ref)
    tol = (HALF[out] + 3.1 * 2.0 ** -24) * np.abs(ref) + 1e-37
    bad = ok & ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], ref[bad][:4])
    assert (got[~ok] == float(torch.tensor(SENTINEL).to(tt(out)))).all()


@pytest.mark.parametrize("counts", COUNTS)
def test_i8_segments(m, counts):
    i8_case(m, counts, 96, 128, extra_rows=3)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("N, K", [(1, 1), (3, 5), (31, 33), (129, 127), (64, 16), (130, 400), (257, 1040), (512, 2048),
                                  (16, 14336)])
def test_i8_sizes(m, N, K, out):
    i8_case(m, [3, 0, 140], N, K, out, seed=N + K)
    i8_case(m, [2, 1, 0], N, K, out, seed=N + K)


@pytest.mark.parametrize("counts", [[1, 0, 63, 64], [65, 128, 129], [255, 256, 257, 0, 5]])
@pytest.mark.parametrize("N, K", [(264, 2064), (1000, 2048), (37, 4000), (37, 4001)])
def test_i8_long_reductions(m, N, K, counts):
    """Large tiles whole and cut (and the other kernel's cuts): sums of parts stay exact."""
    ids = lambda rng, rows: rng.integers(-3, 2 * 70 + 9, rows)
    i8_case(m, counts, N, K, pad=3, extra_rows=9)
    i8_case(m, counts, N, K, out="f32", pad=2, ids=ids, row_div=2, x_rows=70)


def test_i8_lookup(m):
    ids = lambda rng, rows: rng.integers(-4, 3 * 50 + 30, rows)
    i8_case(m, [5, 0, 130, 128], 72, 96, pad=128, ids=ids, row_div=3, x_rows=50)
    i8_case(m, [5, 0, 130, 128], 71, 89, pad=128, ids=ids, row_div=3, x_rows=50)


def test_i8_extreme_codes_do_not_leave_32_bits(m):
    """The longest reduction with every product at its largest, 131071 * 128 * 128 < 2^31."""
    K = 131071
    s = m.make_grouped_shape(2, 1, K, 1, x_dtype="i8", out_dtype="f32")
    q = torch.full((2, K), -128, dtype=torch.int8, device="cuda")
    y = torch.empty(2, 1, dtype=torch.float32, device="cuda")
    one = torch.ones(2, dtype=torch.float32, device="cuda")
    off = dev(np.array([0, 2], dtype=np.int32))
    m.moe_grouped_matmul_i8(s, q, one, None, off, None, q[:1].contiguous().view(1, 1, K), one[:1], y,
                            m.alloc_grouped_workspace(s))
    ref = K * 16384.0
    assert (abs(y.double() - ref) <= ref * 2.0 ** -24).all()


def test_i8_scale_of_a_broken_row(m):
    """A row whose scale is NaN gives NaN in its own products only."""
    x = torch.randn(9, 64, device="cuda")
    x[4, 3] = float("inf")
    q, sc = torch.empty(9, 64, dtype=torch.int8, device="cuda"), torch.empty(9, device="cuda")
    m.moe_quantize_rows(x, q, sc)
    s = m.make_grouped_shape(9, 8, 64, 1, x_dtype="i8", out_dtype="f32")
    y = torch.empty(9, 8, device="cuda")
    m.moe_grouped_matmul_i8(s, q, sc, None, dev(np.array([0, 9], dtype=np.int32)), None,
                            torch.ones(1, 8, 64, dtype=torch.int8, device="cuda"), torch.ones(1, 8, device="cuda"), y,
                            m.alloc_grouped_workspace(s))
    assert torch.isnan(y[4]).all() and torch.isfinite(y[torch.arange(9) != 4]).all()


# ------------------------------------------------- streams, graphs, order --

def test_repeated_calls_give_the_same_bits(m):
    c = Case([300, 0, 5, 129], 260, 1032)
    y, (gx, gw) = c.forward(m), c.backward(m)
    for _ in range(3):
        assert torch.equal(c.forward(m), y)
        hx, hw = c.backward(m)
        assert torch.equal(hx, gx) and torch.equal(hw, gw)


def test_on_another_stream(m):
    c = Case([300, 0, 5, 129], 260, 1032)
    want = c.forward(m)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    s = c.shape(m)
    y = torch.full_like(want, SENTINEL)
    ws = c.ws(m, s)
    st.wait_stream(torch.cuda.current_stream())
    m.moe_grouped_matmul(s, c.x, None, c.offsets, c.counts, c.w, y, ws, stream=st)
    st.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("N, K, many", [(264, 1024, 0), (37, 61, 0), (1288, 1032, 0), (3, 5001, 0), (264, 520, 60)])
def test_captured_into_a_graph(m, N, K, many):
    """Captured once and replayed on new inputs and new tables, with eager work between the replays."""
    ids = lambda rng, rows: rng.permutation(rows)
    c = Case([40, 0, 5, 129] + [0] * many, N, K, extra_rows=60, ids=ids, x_rows=40 + 5 + 129 + 60)
    s = c.shape(m)
    y, gx, gw = c.forward(m), *c.backward(m)
    ws = c.ws(m, s)

    def step():
        m.moe_grouped_matmul(s, c.x, c.ids_t, c.offsets, c.counts, c.w, y, ws)
        m.moe_grouped_matmul_backward(s, c.dy, c.x, c.ids_t, c.offsets, c.counts, c.w, gx, gw, ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    rng = np.random.default_rng(3)
    for i in range(4):
        cnt = rng.integers(0, 58, 4) if not many else rng.integers(0, 4, 4 + many)
        off = np.concatenate([[0], np.cumsum(cnt)])
        c.offsets.copy_(dev(off.astype(np.int32)))
        c.counts.copy_(dev(cnt.astype(np.int32)))
        c.x.normal_()
        c.dy.normal_()
        for t in (y, gx, gw):
            t.fill_(SENTINEL)
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, gx, gw)]
        for t in (y, gx, gw):
            t.fill_(SENTINEL)
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (y, gx, gw))), i


# ------------------------------------------------------- past 32-bit offsets --

def test_weights_past_32_bit_offsets(m):
    """Weights of 2.7e9 elements: the last expert's products, and its gradients."""
    E, N, K = 5, 16384, 32768
    w = torch.empty(E, N, K, dtype=torch.bfloat16, device="cuda").normal_(std=0.05)
    x, dy = torch.randn(3, K, device="cuda").bfloat16(), torch.randn(3, N, device="cuda").bfloat16()
    off, cnt = dev(np.array([0, 0, 0, 0, 0, 3], dtype=np.int32)), dev(np.array([0, 0, 0, 0, 3], dtype=np.int32))
    s = m.make_grouped_shape(3, N, K, E, out_dtype="f32")
    y = torch.empty(3, N, device="cuda")
    ws = m.alloc_grouped_workspace(s)
    m.moe_grouped_matmul(s, x, None, off, cnt, w, y, ws)
    rows = [0, 1, N // 2 + 5, N - 1]
    a, b = x.double().cpu(), w[4][rows].double().cpu()
    assert ((y[:, rows].double().cpu() - a @ b.t()).abs() <= 8 * K ** 0.5 * 2.0 ** -23 * (a.abs() @ b.abs().t())).all()
    s2 = m.make_grouped_shape(3, N, K, E, out_dtype="bf16")
    dx, dw = torch.empty(3, K, dtype=torch.bfloat16, device="cuda"), torch.empty_like(w)
    m.moe_grouped_matmul_backward(s2, dy, x, None, off, cnt, w, dx, dw, m.alloc_grouped_workspace(s2))
    cols = [0, 3, K // 2 + 1, K - 1]
    g, b = dy.double().cpu(), w[4][:, cols].double().cpu()
    ref = g @ b
    assert ((dx[:, cols].double().cpu() - ref).abs()
            <= HALF["bf16"] * ref.abs() + 8 * N ** 0.5 * 2.0 ** -23 * (g.abs() @ b.abs())).all()
    ref = g[:, rows].t() @ a[:, cols]
    got = dw[4][rows][:, cols].double().cpu()
    assert ((got - ref).abs() <= HALF["bf16"] * ref.abs() + 1e-5).all()
    assert (dw[:4].view(torch.int16) == 0).all()


def test_rows_past_32_bit_offsets(m):
    """Rows of 2.2e9 elements on either side of the product."""
    rows, N, K = 140000, 16, 16000
    x = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.empty(2, N, K, dtype=torch.bfloat16, device="cuda").normal_(std=0.05)
    off = dev(np.array([0, 70001, rows], dtype=np.int32))
    pick = [0, 70000, 70001, rows - 1]
    s = m.make_grouped_shape(rows, N, K, 2, out_dtype="f32")
    y = torch.empty(rows, N, device="cuda")
    m.moe_grouped_matmul(s, x, None, off, None, w, y, m.alloc_grouped_workspace(s))
    for r in pick:
        a, b = x[r].double().cpu(), w[int(r > 70000)].double().cpu()
        assert ((y[r].double().cpu() - b @ a).abs() <= 8 * K ** 0.5 * 2.0 ** -23 * (b.abs() @ a.abs())).all(), r
    del y
    # and as the gradient's output
    dy = torch.randn(rows, N, device="cuda").bfloat16()
    dx = x                                              # reuse the memory: dx does not read x
    s2 = m.make_grouped_shape(rows, N, K, 2)
    m.moe_grouped_matmul_backward(s2, dy, None, None, off, None, w, dx, None, m.alloc_grouped_workspace(s2))
    for r in pick:
        g, b = dy[r].double().cpu(), w[int(r > 70000)].double().cpu()
        ref = g @ b
        assert ((dx[r].double().cpu() - ref).abs()
                <= HALF["bf16"] * ref.abs() + 8 * N ** 0.5 * 2.0 ** -23 * (g.abs() @ b.abs())).all(), r


@pytest.mark.parametrize("x, N, K", [("bf16", 67, 61), ("f32", 67, 61), ("bf16", 96, 64), ("bf16", 2048, 2048)])
def test_rows_of_zeros_add_nothing_to_the_weight_gradient(m, x, N, K):
    """Rows whose row_ids name no row of x: NaN and infinities in their dy do not reach dw, on small tiles and on large
    ones, in the first, whole and last stages of a segment."""
    def ids(rng, rows):
        v = rng.integers(0, 40, rows)
        v[::7] = -1
        v[5::11] = 40
        v[:3] = -1
        return v
    c = Case([70, 330], N, K, x, "f32", ids=ids, row_div=1, x_rows=40, seed=N)
    none = (c.ids < 0) | (c.ids >= 40)
    dy = H.to_f64(c.dy)
    dy[none] = 0
    xs = G.lookup(H.to_f64(c.x), c.ids, 1, c.rows)
    rw = G.grouped_matmul_backward(dy, xs, c.segs, H.to_f64(c.w))[1]
    aw = G.grouped_matmul_backward(abs(dy), abs(xs), c.segs, abs(H.to_f64(c.w)))[1]
    at = np.flatnonzero(none)
    c.dy[dev(at[::2])] = float("nan")
    c.dy[dev(at[1::2])] = float("inf")
    close(H.to_f64(c.backward(m, dx=False)[1]), rw, aw, 330, "f32")


@pytest.mark.parametrize("counts, N, K", [([5, 3], 64, 64), ([130, 128], 72, 89), ([130, 128], 37, 4001),
                                          ([130, 128], 264, 2064), ([130, 128], 22016, 64)])
def test_i8_rows_of_zeros_stay_zero(m, counts, N, K):
    """A row that row_ids stands for zeros has the product 0 for scales of infinity and NaN too; a row of x with the
    scale 0 or -0 has the formula's NaN."""
    rows = sum(counts)
    c = Case(counts, 1, 1, "bf16", "f32")
    ids = np.arange(rows, dtype=np.int32) % 8
    ids[::3] = -1
    xs = np.full(8, 0.5, dtype=np.float32)
    xs[4], xs[5] = 0.0, -0.0
    ws = np.full((2, N), np.inf, dtype=np.float32)
    ws[:, ::2] = np.nan
    s = m.make_grouped_shape(rows, N, K, 2, 8, 1, "i8", "f32")
    y = torch.full((rows, N), SENTINEL, dtype=torch.float32, device="cuda")
    one = torch.ones
    m.moe_grouped_matmul_i8(s, one(8, K, dtype=torch.int8, device="cuda"), dev(xs), dev(ids), c.offsets, c.counts,
                            one(2, N, K, dtype=torch.int8, device="cuda"), dev(ws), y, c.ws(m, s))
    y = y.cpu().numpy()
    assert (y[ids < 0] == 0).all()
    assert np.isnan(y[(ids == 4) | (ids == 5)]).all()
    assert np.isnan(y[ids == 0][:, ::2]).all() and np.isposinf(y[ids == 0][:, 1::2]).all()


def test_a_workspace_off_the_gpu_is_refused(m):
    c = Case([5, 3], 64, 64)
    s = c.shape(m)
    y = torch.empty(c.rows, c.N, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="workspace"):
        m.moe_grouped_matmul(s, c.x, None, c.offsets, c.counts, c.w, y, torch.empty(1 << 20, dtype=torch.uint8))
