"""Cases of the layer's separate operators, each in two forms.

The operators are the parts of an MoE layer that a program calls by itself
when its experts are not the fused SwiGLU layer, when it trains, or when it
serves experts held in 8 bits:

  matmul            y[r] = x[row(r)] . w[e]^T for the rows r of expert e's
                    segment of the expert-sorted order
  backward          the gradients of that product: dx[r] = dy[r] . w[e], and
                    dw[e] = sum over the segment of dy[r]^T x[row(r)]
  i8                the same product in 8-bit integers: the activations are
                    quantised with one scale for each token, the weights come
                    with one scale for each output channel
  combine           out[t] = sum_j weights[t, j] * y[inv[t, j]], the way from
                    the expert-sorted order back to the tokens
  combine_backward  its gradients: dy[inv[t, j]] = weights[t, j] * dout[t] and
                    dweights[t, j] = <dout[t], y[inv[t, j]]>

``own`` false computes them with elementary torch operations, true calls the
library.  Nothing here needs the other side.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
_T = {"bf16": torch.bfloat16, "f32": torch.float32}
_B = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------- cases --
# Fields.  T tokens with k of E experts each; `active` experts get rows, the
# others' segments are empty; `skew` is the exponent of the experts'
# popularity (0: even); `pad` the multiple that segments are padded to (1: none;
# 128: the order that moe_route writes, with rows behind each segment that
# belong to nobody); K values in and N out of the product; `gather` whether
# the rows of x are tokens found through the sorted order (the first products
# of a layer) or lie in that order already (the last one).  `x` and `out` are
# the types of the inputs and of y or dw.

def listed():
    return [
        # One token through the first product of a 256-expert layer (the shapes of the Q4_0 batch of
        # one, here in bfloat16): 17 MB of weights, where launch and first loads count.
        dict(name="matmul_one_token", op="matmul", T=1, k=8, E=256, active=8, K=2048, N=512, skew=0.0, pad=1,
             gather=True, x="bf16", out="bf16"),
        # A decode batch of 64 over 64 fine-grained experts, about six rows each: a stream of weights.
        dict(name="matmul_batch64", op="matmul", T=64, k=6, E=64, active=64, K=2048, N=1408, skew=0.3, pad=1,
             gather=True, x="bf16", out="bf16"),
        # The gate product of a 4096-token prompt over 8 wide experts, in moe_route's padded order.
        dict(name="matmul_prompt", op="matmul", T=4096, k=2, E=8, active=8, K=4096, N=14336, skew=1.2, pad=128,
             gather=True, x="bf16", out="bf16"),
        # An fp32 layer of odd sizes with experts that nobody chose (tests of a model, small studies).
        dict(name="matmul_f32_odd", op="matmul", T=333, k=3, E=7, active=5, K=515, N=1003, skew=0.8, pad=1,
             gather=False, x="f32", out="f32"),
        # A training step through the gate product of the wide experts; gradients of the weights in fp32.
        dict(name="backward_prompt", op="backward", T=4096, k=2, E=8, active=8, K=4096, N=14336, skew=1.2, pad=128,
             gather=True, x="bf16", out="f32"),
        # A micro-batch of 1024 tokens over 64 fine-grained experts: short, ragged segments.
        dict(name="backward_fine", op="backward", T=1024, k=6, E=64, active=64, K=2048, N=1408, skew=0.5, pad=1,
             gather=True, x="bf16", out="bf16"),
        # Sizes that are no multiple of anything, an expert with no rows: rows of 834 and 1222 bytes.
        dict(name="backward_odd", op="backward", T=201, k=2, E=9, active=8, K=417, N=611, skew=0.8, pad=1,
             gather=False, x="bf16", out="bf16"),
        # One token through the second product of a layer whose eight experts have 14336 channels.
        dict(name="i8_one_token", op="i8", T=1, k=2, E=8, active=2, K=14336, N=4096, skew=0.0, pad=1,
             gather=False, x="bf16", out="bf16"),
        # The decode batch of 64, with experts in 8 bits.
        dict(name="i8_batch64", op="i8", T=64, k=6, E=64, active=64, K=2048, N=1408, skew=0.3, pad=1,
             gather=True, x="bf16", out="bf16"),
        # The 4096-token prompt, with experts in 8 bits.
        dict(name="i8_prompt", op="i8", T=4096, k=2, E=8, active=8, K=4096, N=14336, skew=1.2, pad=128,
             gather=True, x="bf16", out="bf16"),
        # The prompt's way back to the tokens.
        dict(name="combine_prompt", op="combine", T=4096, k=2, E=8, active=8, N=4096, skew=1.2, pad=128,
             x="bf16", out="bf16"),
        # The training micro-batch's gradients of rows and routing weights.
        dict(name="combine_backward_fine", op="combine_backward", T=1024, k=6, E=64, active=64, N=2048, skew=0.5,
             pad=1, x="bf16", out="bf16"),
    ]


_MAX_FLOPS = 4.0 * 8192 * 4096 * 14336      # backward_prompt
_MAX_WEIGHTS = 8 * 4096 * 14336


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A size of [lo, hi], spread over its logarithm: half of them multiples of 64, the others any."""
    n = _log(rng, lo, hi)
    if rng.random() < 0.5:
        n = max(64, (n + 32) // 64 * 64)
    return max(lo, min(n, hi))


def draw(rng):
    while True:
        op = rng.choice(["matmul", "matmul", "backward", "backward", "i8", "i8", "combine", "combine_backward"])
        E = _log(rng, 1, 256)
        k = rng.randint(1, min(8, E))
        T = _log(rng, 1, 4096)
        active = rng.randint(k, min(E, T * k))
        c = dict(op=op, T=T, k=k, E=E, active=active, skew=rng.choice([0.0, 0.5, 1.2]),
                 pad=rng.choice([1, 1, 128]) if T > 64 else 1)
        if op in ("matmul", "backward", "i8"):
            c["K"], c["N"] = _size(rng, 32, 14336), _size(rng, 32, 14336)
            c["gather"] = rng.random() < 0.5
            c["x"] = "bf16" if op == "i8" or rng.random() < 0.75 else "f32"
            c["out"] = c["x"] if c["x"] == "f32" or rng.random() < 0.7 else "f32"
            # fp32 products run at an eighth of the bfloat16 rate or less: smaller ones are drawn
            if work(c)["flops"] > _MAX_FLOPS / (32 if c["x"] == "f32" else 2):
                continue
            if E * c["K"] * c["N"] > _MAX_WEIGHTS // 2:
                continue
        else:
            c["N"] = _size(rng, 32, 8192)
            c["x"] = rng.choice(["bf16", "bf16", "f32"])
            c["out"] = rng.choice(["bf16", "f32"])
            if work(c)["bytes"] > 400e6:
                continue
        return c


def work(case):
    """Bytes and operations that the pass cannot do without: each engaged
    expert's weights, each row, table entry and output once."""
    c = case
    M, N, x, o = c["T"] * c["k"], c["N"], _B[c["x"]], _B[c["out"]]
    if c["op"] == "combine":
        return {"bytes": M * N * x + M * 8 + c["T"] * N * o, "flops": 2 * M * N}
    if c["op"] == "combine_backward":
        return {"bytes": 2 * M * N * x + c["T"] * N * o + M * 12, "flops": 3 * M * N}
    K = c["K"]
    rows_in = c["T"] if c["gather"] else M
    tables = (2 * c["E"] + 1) * 4 + (M * 4 if c["gather"] else 0)
    if c["op"] == "matmul":
        return {"bytes": c["active"] * N * K * x + rows_in * K * x + M * N * o + tables, "flops": 2 * M * N * K}
    if c["op"] == "i8":
        return {"bytes": c["active"] * (N * K + 4 * N) + rows_in * K * x + M * N * o + tables, "flops": 2 * M * N * K}
    return {"bytes": c["active"] * N * K * x + rows_in * K * x + M * N * x + M * K * x + c["E"] * N * K * o + tables,
            "flops": 4 * M * N * K}


# ------------------------------------------------------------------ inputs --

def _routing(c, seed):
    """Expert-sorted order of a routing in which exactly `active` experts get rows: per-token distinct
    experts by popularity, after the first tokens have taken each expert in turn."""
    g = torch.Generator().manual_seed(seed * 7919 + 17)
    T, k, E, active, pad = c["T"], c["k"], c["E"], c["active"], c["pad"]
    chosen = torch.sort(torch.randperm(E, generator=g)[:active]).values
    order = torch.randperm(active, generator=g)
    logp = -c["skew"] * torch.log(torch.arange(1, active + 1, dtype=torch.float64))
    gumbel = -torch.log(-torch.log(torch.rand(T, active, generator=g, dtype=torch.float64).clamp(1e-12, 1 - 1e-12)))
    local = torch.topk(logp + gumbel, k, dim=1).indices
    first = min(T, (active + k - 1) // k)
    local[:first] = (torch.arange(first * k) % active).view(first, k)
    ids = chosen[order[local]].reshape(-1)                              # [T*k], expert of assignment f = t*k + j
    M = T * k
    counts = torch.bincount(ids, minlength=E)
    padded = (counts + pad - 1) // pad * pad
    offsets = torch.zeros(E + 1, dtype=torch.int64)
    offsets[1:] = torch.cumsum(padded, 0)
    rows = M if pad == 1 else (M + E * (pad - 1) + pad - 1) // pad * pad
    by_expert = torch.sort(ids, stable=True).indices                    # assignments in expert order
    start = torch.cumsum(counts, 0) - counts
    e_of = ids[by_expert]
    pos = offsets[e_of] + (torch.arange(M) - start[e_of])               # their sorted rows
    sorted_ids = torch.full((rows,), M, dtype=torch.int64)
    sorted_ids[pos] = by_expert
    inv = torch.empty(M, dtype=torch.int64)
    inv[by_expert] = pos
    i32 = lambda a: a.to(torch.int32).to(DEV)
    return dict(rows=rows, counts_host=counts.tolist(), offsets_host=offsets.tolist(), counts=i32(counts),
                offsets=i32(offsets), sorted_ids=i32(sorted_ids), inv=i32(inv))


def _randn(g, shape, dtype, scale=1.0):
    """Normal values, drawn in pieces along the first axis (a stack of weights is large in 32 bits)."""
    out = torch.empty(shape, dtype=dtype, device=DEV)
    for i in range(0, shape[0], max(1, (1 << 26) // max(1, out[0].numel()))):
        piece = out[i:i + max(1, (1 << 26) // max(1, out[0].numel()))]
        piece.copy_(torch.randn(piece.shape, generator=g, device=DEV) * scale)
    return out


def _codes(g, shape):
    """8-bit codes of normal weights whose row's largest is about four deviations."""
    out = torch.empty(shape, dtype=torch.int8, device=DEV)
    for i in range(shape[0]):
        out[i].copy_((torch.randn(shape[1:], generator=g, device=DEV) * 32).round_().clamp_(-127, 127))
    return out


def _inputs(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case=c, **_routing(c, seed))
    xt, rows, N = _T[c["x"]], s["rows"], c["N"]
    if c["op"] in ("combine", "combine_backward"):
        s["y"] = _randn(g, (rows, N), xt)
        s["weights"] = torch.softmax(torch.randn(c["T"], c["k"], generator=g, device=DEV), dim=1).reshape(-1)
        if c["op"] == "combine_backward":
            s["dout"] = _randn(g, (c["T"], N), _T[c["out"]])
        return s
    K = c["K"]
    s["x"] = _randn(g, (c["T"] if c["gather"] else rows, K), xt)
    if c["op"] == "i8":
        # a few channels of activations are far larger than the others
        loud = torch.rand(K, generator=g, device=DEV) < 0.01
        s["x"].mul_(torch.where(loud, 12.0, 1.0).to(xt))
        s["w"] = _codes(g, (c["E"], N, K))
        s["w_scale"] = 6e-4 * (0.5 + torch.rand(c["E"], N, generator=g, device=DEV))
    else:
        s["w"] = _randn(g, (c["E"], N, K), xt, 0.02)
    if c["op"] == "backward":
        s["dy"] = _randn(g, (rows, N), xt)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    c, rows = case, s["rows"]
    N, xt, ot = c["N"], _T[c["x"]], _T[c["out"]]
    # buffers that a program keeps; rows that belong to no expert stay as they are (zero)
    if c["op"] in ("matmul", "i8"):
        s["res"] = [torch.zeros(rows, N, dtype=ot, device=DEV)]
    elif c["op"] == "backward":
        s["res"] = [torch.zeros(rows, c["K"], dtype=xt, device=DEV),
                    torch.zeros(c["E"], N, c["K"], dtype=ot, device=DEV)]
    elif c["op"] == "combine":
        s["res"] = [torch.zeros(c["T"], N, dtype=ot, device=DEV)]
    else:
        s["res"] = [torch.zeros(rows, N, dtype=xt, device=DEV),
                    torch.zeros(c["T"] * c["k"], dtype=torch.float32, device=DEV)]
    if own:
        import mixture_experts_layer_12_amd as m
        s["m"] = m
        if c["op"] in ("combine", "combine_backward"):
            s["shape"] = m.make_combine_shape(T=c["T"], top_k=c["k"], H=N, rows=rows, y_dtype=c["x"],
                                              out_dtype=c["out"])
        else:
            xr, div = (c["T"], c["k"]) if c["gather"] else (rows, 1)
            s["shape"] = m.make_grouped_shape(rows=rows, N=N, K=c["K"], E=c["E"], x_rows=xr, row_div=div,
                                              x_dtype="i8" if c["op"] == "i8" else c["x"], out_dtype=c["out"])
            s["ws"] = m.alloc_grouped_workspace(s["shape"], DEV)
            if c["op"] == "i8":
                s["xq"] = torch.empty(s["x"].shape, dtype=torch.int8, device=DEV)
                s["x_scale"] = torch.empty(s["x"].shape[0], dtype=torch.float32, device=DEV)
    return s


# -------------------------------------------------------------------- runs --

def run(state):
    s = state
    return (_run_own if own else _run_plain)(s, s["case"]["op"])


def _run_own(s, op):
    m, res = s["m"], s["res"]
    if op == "combine":
        m.moe_combine(s["shape"], s["y"], s["inv"], s["weights"], res[0])
        return res
    if op == "combine_backward":
        m.moe_combine_backward(s["shape"], s["dout"], s["y"], s["inv"], s["weights"], res[0], res[1])
        return res
    ids = s["sorted_ids"] if s["case"]["gather"] else None
    if op == "matmul":
        m.moe_grouped_matmul(s["shape"], s["x"], ids, s["offsets"], s["counts"], s["w"], res[0], s["ws"])
    elif op == "backward":
        m.moe_grouped_matmul_backward(s["shape"], s["dy"], s["x"], ids, s["offsets"], s["counts"], s["w"],
                                      res[0], res[1], s["ws"])
    else:
        m.moe_quantize_rows(s["x"], s["xq"], s["x_scale"])
        m.moe_grouped_matmul_i8(s["shape"], s["xq"], s["x_scale"], ids, s["offsets"], s["counts"], s["w"],
                                s["w_scale"], res[0], s["ws"])
    return res


def _segments(s):
    for e, n in enumerate(s["counts_host"]):
        if n:
            yield e, s["offsets_host"][e], s["offsets_host"][e] + n


def _run_plain(s, op):
    c, res = s["case"], s["res"]
    if op == "combine":
        picked = s["y"][s["inv"].long()].float().view(c["T"], c["k"], c["N"])
        res[0].copy_((picked * s["weights"].view(c["T"], c["k"], 1)).sum(dim=1))
        return res
    if op == "combine_backward":
        inv, dout = s["inv"].long(), s["dout"].float().unsqueeze(1)
        picked = s["y"][inv].float().view(c["T"], c["k"], c["N"])
        res[0][inv] = (dout * s["weights"].view(c["T"], c["k"], 1)).to(res[0].dtype).view(-1, c["N"])
        res[1].copy_((picked * dout).sum(dim=2).view(-1))
        return res
    ids = torch.div(s["sorted_ids"], c["k"], rounding_mode="floor") if c["gather"] else None
    rows_of = lambda a, b: ids[a:b] if c["gather"] else slice(a, b)
    if op == "matmul":
        for e, a, b in _segments(s):
            res[0][a:b] = (s["x"][rows_of(a, b)].float() @ s["w"][e].float().t()).to(res[0].dtype)
    elif op == "backward":
        for e, n in enumerate(s["counts_host"]):
            a = s["offsets_host"][e]
            b = a + n
            dy = s["dy"][a:b].float()
            res[0][a:b] = (dy @ s["w"][e].float()).to(res[0].dtype)
            res[1][e] = (dy.t() @ s["x"][rows_of(a, b)].float()).to(res[1].dtype)
    else:
        # the scale is the row's largest magnitude over 127, rounded to 32 bits; the code the nearest
        # whole number of the quotient, found in 64 bits because a half decides it; the sums of
        # products of codes pass 24 bits
        x = s["x"].double()
        scale = (x.abs().amax(dim=1, keepdim=True) / 127).float()
        codes = torch.where(scale > 0, torch.round(x / scale.double()), 0.0).clamp_(-127, 127)
        for e, a, b in _segments(s):
            r = rows_of(a, b)
            acc = (codes[r] @ s["w"][e].double().t()).float()
            res[0][a:b] = (acc * scale[r] * s["w_scale"][e]).to(res[0].dtype)
    return res


# ------------------------------------------------------------------- exact --

def exact(case, seed):
    c = case
    s = _inputs(c, seed)
    N, rows, M = c["N"], s["rows"], c["T"] * c["k"]
    f64 = dict(dtype=torch.float64, device=DEV)
    inv = s["inv"].long()
    token = torch.arange(M, device=DEV) // c["k"]
    if c["op"] == "combine":
        out = torch.zeros(c["T"], N, **f64)
        for j in range(c["k"]):
            out += s["weights"].double()[j::c["k"], None] * s["y"].double().index_select(0, inv[j::c["k"]])
        return [out]
    if c["op"] == "combine_backward":
        dy, dw = torch.zeros(rows, N, **f64), torch.zeros(M, **f64)
        for j in range(c["k"]):
            at = inv[j::c["k"]]
            dy.index_copy_(0, at, s["weights"].double()[j::c["k"], None] * s["dout"].double())
            dw[j::c["k"]] = (s["dout"].double() * s["y"].double().index_select(0, at)).sum(1)
        return [dy, dw]
    # the expert of each assignment, from the tables; assignments (not sorted rows) are walked
    expert = torch.bucketize(inv, s["offsets"].long()[1:], right=True)
    source = token if c["gather"] else inv
    if c["op"] == "i8":
        x = s["x"].double()
        scale = (x.abs().max(dim=1).values / 127.0).float().double()
        safe = torch.where(scale > 0, scale, 1.0)
        x = torch.round(x / safe[:, None]).clamp(-127, 127)
        x = x * scale[:, None]
    else:
        x = s["x"]
    y = torch.zeros(rows, N, **f64) if c["op"] != "backward" else None
    dx = torch.zeros(rows, c["K"], **f64) if c["op"] == "backward" else None
    dw = torch.zeros(c["E"], N, c["K"], **f64) if c["op"] == "backward" else None
    for e in torch.unique(expert).tolist():
        f = (expert == e).nonzero().view(-1)
        w = s["w"][e].double()
        xe = x.index_select(0, source[f]).double()
        if c["op"] == "backward":
            g = s["dy"].index_select(0, inv[f]).double()
            dx.index_copy_(0, inv[f], torch.mm(g, w))
            torch.mm(g.t(), xe, out=dw[e])
        else:
            if c["op"] == "i8":
                w = w * s["w_scale"][e].double()[:, None]
            y.index_copy_(0, inv[f], torch.mm(xe, w.t()))
    return [dx, dw] if c["op"] == "backward" else [y]
