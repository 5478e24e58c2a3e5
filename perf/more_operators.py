"""The operators of an expert layer in 8-bit integers, as cases to measure: products of int8 operands
with a scale for each token and each channel, the quantisation that makes such operands (rows
gathered by index, or joined with their gate), and tokens sorted by expert and back, weighted, with
the gradients of both ways.

With `own` false, run() computes them from elementary torch operations; with `own` true it calls
the library's entry points (include/htint8.h, include/htroute.h).
"""
import math
import types

import torch

own = False

INT8_MAX = 127.0
MIN_SCALE = 2.0 ** -126

# Sizes a draw stays within; the largest product is the benchmark's 8192^3, the largest exchange of
# tokens 16384 of 4096 values to 8 experts each.
MOST_FLOPS = 2 * 8192 ** 3
MOST_MOVED = 16384 * 8 * 4096


# ---- cases ---------------------------------------------------------------------------------

def listed():
    return [
        # one token through one linear layer: latency
        product("product 1x4096x4096", 1, 4096, 4096, bias=True),
        # a decode batch against a wide weight: the weight's bytes bound it
        product("product 16x16384x8192", 16, 16384, 8192),
        # a short prompt, every size off the tiles' and the loads' widths, bias and activation
        product("product 333x4001x8190 f16", 333, 4001, 8190, out="f16", bias=True, act="gelu"),
        # a large prefill step
        product("product 8192x8192x8192", 8192, 8192, 8192),
        # a prompt through an expert layer's product
        experts("experts prefill 8190 of 32", 8190, 32, 4096, 2048),
        # one token's activations before a product
        quant("quantise 1x8192 bf16", 1, 8192, "bf16"),
        # a prefill batch's activations
        quant("quantise 16384x8192 bf16", 16384, 8192, "bf16"),
        # a decode batch to its experts' rows, and the way back of the gradient; an odd width
        sort("sort 37x2051 f16, 6 of 64", 37, 2051, 64, 6, 1, "f16"),
        # a training batch to its experts' rows, groups aligned for the weight gradient
        sort("sort 16384x4096 8 of 256", 16384, 4096, 256, 8, 16, "bf16"),
        # a decode batch's rows joined by their gates, with the gradients
        combine("combine 37x2051 f32, 6 of 64", 37, 2051, 64, 6, 1, "f32", "f32"),
        # a training batch's rows joined by their gates, with the gradients
        combine("combine 16384x4096 8 of 256", 16384, 4096, 256, 8, 16, "bf16", "f32"),
        # a decode batch through a whole expert layer: quantised by expert, two products with the
        # gated activation between them, and joined
        layer("layer 64 tokens 8 of 64", 64, 2048, 1024, 64, 8),
    ]


def product(name, M, N, K, out="bf16", bias=False, act="none", accumulate=False, dense=False):
    # dense: rows of K codes directly behind each other, else padded to 16 bytes
    return {"name": name, "kind": "product", "M": M, "N": N, "K": K, "out": out, "bias": bias, "act": act,
            "accumulate": accumulate, "dense": dense}


def experts(name, rows, E, N, K, act="none"):
    return {"name": name, "kind": "experts", "rows": rows, "E": E, "N": N, "K": K, "act": act}


def quant(name, rows, cols, dtype, gather=0):
    return {"name": name, "kind": "quant", "rows": rows, "cols": cols, "dtype": dtype, "gather": gather}


def sort(name, tokens, H, E, topk, align, dtype):
    return {"name": name, "kind": "sort", "tokens": tokens, "H": H, "E": E, "topk": topk, "align": align, "dtype": dtype}


def combine(name, tokens, H, E, topk, align, dtype, weight):
    return {"name": name, "kind": "combine", "tokens": tokens, "H": H, "E": E, "topk": topk, "align": align,
            "dtype": dtype, "weight": weight}


def layer(name, tokens, H, F, E, topk):
    return {"name": name, "kind": "layer", "tokens": tokens, "H": H, "F": F, "E": E, "topk": topk}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["product", "product", "product", "experts", "experts", "quant", "quant", "sort", "sort",
                       "combine", "combine", "layer"])
    if kind == "product":
        while True:
            M, N, K = _log(rng, 1, 8192), _log(rng, 256, 16384), _log(rng, 128, 8192)
            if rng.random() < 0.7:
                K = _up(K, 16)
            if 2 * M * N * K <= MOST_FLOPS:
                break
        c = product("", M, N, K, out=rng.choice(["bf16", "bf16", "f16", "f32"]), bias=rng.random() < 0.5,
                    act=rng.choice(["none", "relu", "gelu", "silu"]), accumulate=rng.random() < 0.2,
                    dense=rng.random() < 0.3)
    elif kind == "experts":
        while True:
            rows, E, N, K = _log(rng, 8, 16384), _log(rng, 4, 128), 8 * _log(rng, 32, 1024), 16 * _log(rng, 16, 512)
            if 2 * rows * N * K <= MOST_FLOPS / 4 and E * N * K <= 1 << 30:
                break
        c = experts("", rows, E, N, K, act=rng.choice(["none", "silu"]))
    elif kind == "quant":
        rows, cols = _log(rng, 1, 32768), _log(rng, 64, 32768)
        if rows * cols > 1 << 27:
            rows = (1 << 27) // cols
        c = quant("", rows, cols, rng.choice(["bf16", "f16", "f32"]), gather=rng.choice([0, 0, 2, 8]))
    elif kind in ("sort", "combine"):
        while True:
            tokens, E, H, topk = _log(rng, 1, 16384), _log(rng, 4, 256), _log(rng, 64, 8192), rng.randint(1, 8)
            dtype, align = rng.choice(["bf16", "bf16", "f16", "f32"]), rng.choice([1, 16, 128])
            if rng.random() < 0.7:
                H = _up(H, 8)
            if topk <= E and (tokens * topk + E * (align - 1)) * H * _SIZE[dtype] <= 2 * MOST_MOVED:
                break
        c = (sort("", tokens, H, E, topk, align, dtype) if kind == "sort" else
             combine("", tokens, H, E, topk, align, dtype, rng.choice(["f32", dtype])))
    else:
        while True:
            T, H, F = _log(rng, 1, 4096), 16 * _log(rng, 16, 256), 16 * _log(rng, 8, 256)
            E = _log(rng, 4, 64)
            if E * H * F <= 1 << 28 and T * H * F <= 1 << 33:
                break
        c = layer("", T, H, F, E, rng.randint(1, min(8, E)))
    del c["name"]
    return c


def _hit(rows, E):
    """Experts that at least one of `rows` evenly spread rows goes to."""
    return E * (1.0 - (1.0 - 1.0 / E) ** rows)


def _up(n, m):
    return -(-n // m) * m


_SIZE = {"bf16": 2, "f16": 2, "f32": 4}
_TYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def work(case):
    kind = case["kind"]
    if kind == "product":
        M, N, K, size = case["M"], case["N"], case["K"], _SIZE[case["out"]]
        b = M * K + N * K + 4 * (M + N) + M * N * size
        b += (N * size if case["bias"] else 0) + (M * N * size if case["accumulate"] else 0)
        return {"bytes": b, "flops": 2 * M * N * K}
    if kind == "experts":
        R, E, N, K = case["rows"], case["E"], case["N"], case["K"]
        return {"bytes": int(R * K + _hit(R, E) * N * (K + 4) + 4 * R + 2 * R * N + 4 * (E + 1)), "flops": 2 * R * N * K}
    if kind == "quant":
        n = case["rows"] * case["cols"]
        return {"bytes": n // max(1, case["gather"]) * _SIZE[case["dtype"]] + n + 4 * case["rows"], "flops": 3 * n}
    T, H, E, k = case["tokens"], case["H"], case["E"], case["topk"]
    if kind == "layer":
        F, hit, R = case["F"], _hit(T * k, E), T * k
        return {"bytes": int(2 * 2 * T * H + hit * (3 * H * F + 4 * (2 * F + H)) + 12 * R), "flops": 6 * R * H * F}
    live, size = (T - T // 16) * k, _SIZE[case["dtype"]]
    rows = T * k + E * (case["align"] - 1)
    if kind == "sort":      # the tokens and their rows, and both gradients
        return {"bytes": (2 * T + live + rows) * H * size + 4 * (rows + T * k), "flops": live * H}
    # rows and the outputs' gradient, outputs, the rows' and the weights' gradients
    return {"bytes": (live + 2 * T + rows) * H * size + 4 * (rows + T * k) + 2 * T * k * _SIZE[case["weight"]],
            "flops": 5 * live * H}


# ---- inputs --------------------------------------------------------------------------------

def _activations(g, rows, cols):
    """Normal values whose columns differ in size, a few by a lot."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    return x * torch.exp(0.7 * torch.randn(cols, generator=g, device="cuda"))


def _weights(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda") * shape[-1] ** -0.5


def _quantised(x):
    """int8 codes of x (..., cols) and the scale of each row, in float32 with one rounding for each
    operation.  A row with a value that is not finite has scale NaN and codes of zero."""
    x = x.float()
    top = x.abs().amax(-1)
    bad = ~torch.isfinite(top)
    t = top.masked_fill(bad, 0).clamp(min=INT8_MAX * MIN_SCALE)
    most = torch.full_like(t, INT8_MAX)
    q = torch.round(x * (most / t)[..., None]).clamp(-INT8_MAX, INT8_MAX)
    q = q.masked_fill(bad[..., None], 0).to(torch.int8)
    return q, (t / most).masked_fill(bad, math.nan)


def _pitched(q, pitch):
    """The same codes with `pitch` bytes from one row to the next, some other codes between the rows."""
    room = torch.full((q.shape[0], pitch), 85, dtype=torch.int8, device="cuda")
    room[:, : q.shape[1]] = q
    return room[:, : q.shape[1]]


def _sizes(g, rows, E):
    """Where each expert's rows start, from one draw of an expert for each row, some preferred."""
    lean = torch.exp(0.5 * torch.randn(E, generator=g, device="cuda"))
    to = torch.multinomial(lean, rows, replacement=True, generator=g)
    starts = [0]
    for n in torch.bincount(to, minlength=E).tolist():
        starts.append(starts[-1] + n)
    return starts


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = types.SimpleNamespace(**case)
    globals()["_prepare_" + case["kind"]](s, g)
    if own:
        # the handle and the workspace that a program makes once for its sizes
        plan = globals().get("_plan_" + case["kind"])
        if plan:
            plan(s)
    return s


def _make(*sizes, **layout):
    from hierarchical_tiling_amd import htint8
    gemm = htint8.Int8Gemm(htint8.make_desc(*sizes, **layout))
    return gemm, torch.empty(gemm.workspace_bytes, dtype=torch.uint8, device="cuda")


def _prepare_product(s, g):
    s.pitch = s.K if s.dense else _up(s.K, 16)
    q, s.a_scale = _quantised(_activations(g, s.M, s.K))
    s.a = _pitched(q, s.pitch)
    q, s.b_scale = _quantised(_weights(g, s.N, s.K))
    s.b = _pitched(q, s.pitch)
    s.out_type = _TYPE[s.out]
    s.bias_v = (0.1 * torch.randn(s.N, generator=g, device="cuda")).to(s.out_type) if s.bias else None
    s.c = torch.randn(s.M, s.N, generator=g, device="cuda").to(s.out_type) if s.accumulate else None
    s.d = torch.empty(s.M, s.N, dtype=s.out_type, device="cuda")


def _plan_product(s):
    s.gemm, s.workspace = _make(s.M, s.N, s.K, s.out, lda=s.pitch, ldb=s.pitch, ldd=s.N,
                                ldc=s.N if s.accumulate else 0, bias=s.bias, act=s.act)


def _prepare_experts(s, g):
    starts = _sizes(g, s.rows, s.E)
    s.cap = max(b - a for a, b in zip(starts, starts[1:]))
    s.offsets = torch.tensor(starts, dtype=torch.int32, device="cuda")
    s.a, s.a_scale = _quantised(_activations(g, s.rows, s.K))
    s.b, s.b_scale = _quantised(_weights(g, s.E, s.N, s.K))
    s.d = torch.empty(s.rows, s.N, dtype=torch.bfloat16, device="cuda")


def _plan_experts(s):
    s.gemm, s.workspace = _make(s.rows, s.N, s.K, "bf16", lda=s.K, ldb=s.K, ldd=s.N, act=s.act, groups="rows",
                                batch=s.E, b_stride_l=s.N * s.K, b_scale_l=s.N)


def _prepare_quant(s, g):
    # gather > 0: each source row goes to about `gather` rows of the result, in a shuffled order
    # with a few empty places, as tokens go to their experts' rows
    source = max(1, s.rows // max(1, s.gather))
    s.x = _activations(g, source, s.cols).to(_TYPE[s.dtype])
    s.index = None
    if s.gather:
        s.index = torch.randint(-s.gather, source * s.gather, (s.rows,), generator=g, device="cuda", dtype=torch.int32)
    s.q = torch.zeros(s.rows, _up(s.cols, 16), dtype=torch.int8, device="cuda")[:, : s.cols]
    s.scale = torch.empty(s.rows, device="cuda")


def _prepare_exchange(s, g):
    """A routing: gates (tokens, topk), order, slot and offsets, the last sixteenth of the tokens
    being padding that goes nowhere."""
    T, E, k, align = s.tokens, s.E, s.topk, getattr(s, "align", 1)
    logits = torch.randn(T, E, generator=g, device="cuda") + 0.7 * torch.randn(E, generator=g, device="cuda")
    top = logits.topk(k, dim=1)
    s.gates = torch.softmax(top.values, 1)
    live = torch.arange(T, device="cuda") < T - T // 16
    flat = torch.where(live[:, None], top.indices, E).flatten()
    counts = torch.bincount(flat, minlength=E + 1)
    starts = torch.cumsum(counts, 0) - counts
    groups = (counts[:E] + align - 1) // align * align
    s.offsets = torch.cat([torch.zeros_like(groups[:1]), torch.cumsum(groups, 0)]).int()
    by_expert = torch.argsort(flat, stable=True)
    to = flat[by_expert]
    place = torch.arange(T * k, device="cuda") - starts[to] + s.offsets[to]
    place = torch.where(to < E, place, -1)
    s.slot = torch.empty(T * k, dtype=torch.int32, device="cuda")
    s.slot[by_expert] = place.int()
    s.slot = s.slot.view(T, k)
    s.places = T * k + E * (align - 1)
    order = torch.full((s.places + 1,), -1, dtype=torch.int32, device="cuda")
    order[place] = by_expert.int()              # place -1 is the extra last entry
    order[s.places] = -1
    s.order = order[: s.places].clone()
    s.cap = int(counts[:E].max())


def _prepare_sort(s, g):
    _prepare_exchange(s, g)
    dtype = _TYPE[s.dtype]
    s.x = _activations(g, s.tokens, s.H).to(dtype)
    s.d_y = torch.randn(s.places, s.H, generator=g, device="cuda").to(dtype)
    s.y, s.d_x = torch.empty_like(s.d_y), torch.empty_like(s.x)


def _prepare_combine(s, g):
    _prepare_exchange(s, g)
    dtype = _TYPE[s.dtype]
    s.gates = s.gates.to(_TYPE[s.weight])
    s.y = torch.randn(s.places, s.H, generator=g, device="cuda").to(dtype)
    s.d_out = torch.randn(s.tokens, s.H, generator=g, device="cuda").to(dtype)
    s.out, s.d_y, s.d_gates = torch.empty_like(s.d_out), torch.empty_like(s.y), torch.empty_like(s.gates)


def _prepare_layer(s, g):
    _prepare_exchange(s, g)
    T, H, F, E, R = s.tokens, s.H, s.F, s.E, s.places
    s.x = _activations(g, T, H).to(torch.bfloat16)
    s.w1, s.w1_scale = _quantised(_weights(g, E, 2 * F, H))      # the gate's channels, then the others
    s.w2, s.w2_scale = _quantised(_weights(g, E, H, F))
    s.a, s.a_scale = torch.empty(R, H, dtype=torch.int8, device="cuda"), torch.empty(R, device="cuda")
    s.b, s.b_scale = torch.empty(R, F, dtype=torch.int8, device="cuda"), torch.empty(R, device="cuda")
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    s.h, s.y, s.out = torch.zeros(R, 2 * F, **bf16), torch.zeros(R, H, **bf16), torch.empty(T, H, **bf16)


def _plan_layer(s):
    H, F, E, R = s.H, s.F, s.E, s.places
    s.up, s.up_ws = _make(R, 2 * F, H, "bf16", lda=H, ldb=H, ldd=2 * F, groups="rows", batch=E,
                          b_stride_l=2 * F * H, b_scale_l=2 * F)
    s.down, s.down_ws = _make(R, H, F, "bf16", lda=F, ldb=F, ldd=H, groups="rows", batch=E,
                              b_stride_l=H * F, b_scale_l=H)


# ---- one pass ------------------------------------------------------------------------------

def run(s):
    return globals()[("_own_" if own else "_plain_") + s.kind](s)


def _own_product(s):
    s.gemm.run(s.a, s.a_scale, s.b, s.b_scale, s.d, C=s.c, bias=s.bias_v, beta=1.0 if s.accumulate else 0.0,
               workspace=s.workspace)
    return s.d


def _own_experts(s):
    s.gemm.run(s.a, s.a_scale, s.b, s.b_scale, s.d, offsets=s.offsets, workspace=s.workspace)
    return s.d


def _own_quant(s):
    from hierarchical_tiling_amd import htint8
    htint8.quantize(s.x, s.q, s.scale, row_index=s.index, index_div=max(1, s.gather))
    return s.q, s.scale


def _own_sort(s):
    from hierarchical_tiling_amd import htroute
    htroute.gather(s.x, s.order, s.slot, s.y)
    htroute.combine(s.d_y, s.slot, s.d_x)
    return s.y, s.d_x


def _own_combine(s):
    from hierarchical_tiling_amd import htroute
    htroute.combine(s.y, s.slot, s.out, weights=s.gates)
    htroute.combine_grad(s.d_out, s.y, s.order, s.slot, s.gates, s.d_y, s.d_gates)
    return s.out, s.d_y, s.d_gates


def _own_layer(s):
    from hierarchical_tiling_amd import htint8, htroute
    htint8.quantize(s.x, s.a, s.a_scale, row_index=s.order, index_div=s.topk)
    s.up.run(s.a, s.a_scale, s.w1, s.w1_scale, s.h, offsets=s.offsets, workspace=s.up_ws)
    htint8.quantize(s.h[:, s.F:], s.b, s.b_scale, gate=s.h[:, : s.F], act="silu")
    s.down.run(s.b, s.b_scale, s.w2, s.w2_scale, s.y, offsets=s.offsets, workspace=s.down_ws)
    htroute.combine(s.y, s.slot, s.out, weights=s.gates)
    return s.out


def _activate(y, act):
    if act == "relu":
        return y.clamp(min=0)
    if act == "gelu":
        return 0.5 * y * (1 + torch.erf(y * 0.5 ** 0.5))
    if act == "silu":
        return y / (1 + torch.exp(-y))
    return y


def _plain_product(s):
    # sums of codes' products stay below 2^24 on such inputs: float32 holds them
    y = (s.a.float() @ s.b.float().t()) * s.a_scale[:, None] * s.b_scale
    if s.c is not None:
        y = y + s.c.float()
    if s.bias_v is not None:
        y = y + s.bias_v.float()
    return _activate(y, s.act).to(s.out_type)


def _groups(offsets, cap, rows):
    """Rows in groups to a place of their own in (E, cap): group and index within it, and whether a
    row is of any group."""
    row = torch.arange(rows, device="cuda")
    E = offsets.numel() - 1
    group = (row[:, None] >= offsets[None, 1:]).sum(1)
    inside = group < E
    group = group.clamp(max=E - 1)
    return group, (row - offsets[group]).clamp(max=max(cap - 1, 0)), inside


def _plain_rows(a, a_scale, w, w_scale, offsets, cap, act="none"):
    """(rows, N) in float32: each row of codes times its group's matrix; zero outside the groups."""
    group, at, inside = _groups(offsets, cap, a.shape[0])
    x = torch.zeros(w.shape[0], max(cap, 1), a.shape[1], device="cuda")
    x.index_put_((group, at), a.float() * inside[:, None], accumulate=True)
    y = torch.bmm(x, w.float().transpose(1, 2).contiguous())[group, at]
    y = _activate(y * a_scale[:, None] * w_scale[group], act)
    return torch.where(inside[:, None], y, 0.0)


def _plain_experts(s):
    return _plain_rows(s.a, s.a_scale, s.b, s.b_scale, s.offsets, s.cap, s.act).to(torch.bfloat16)


def _gathered(x, index, div):
    """Rows index // div of x; zeros where the index is below zero."""
    return torch.where((index >= 0)[:, None], x[(index.clamp(min=0) // div).long()], 0.0)


def _plain_quant(s):
    return _quantised(s.x if s.index is None else _gathered(s.x.float(), s.index, s.gather))


def _joined(y, slot, weights=None):
    """The sum over each token's rows, float32, weighted if asked; dropped assignments add nothing."""
    rows = torch.where((slot >= 0)[..., None], y.float()[slot.clamp(min=0).long()], 0.0)     # (T, topk, H)
    return (rows if weights is None else rows * weights.float()[..., None]).sum(1)


def _plain_sort(s):
    return _gathered(s.x, s.order, s.topk), _joined(s.d_y, s.slot).to(s.x.dtype)


def _plain_combine(s):
    out = _joined(s.y, s.slot, s.gates)
    at = s.slot.clamp(min=0).long()
    d = s.d_out.float()
    d_gates = torch.where(s.slot >= 0, (s.y.float()[at] * d[:, None, :]).sum(2), 0.0)
    from_ = s.order.clamp(min=0).long()
    d_y = torch.where((s.order >= 0)[:, None], d[from_ // s.topk] * s.gates.float().flatten()[from_][:, None], 0.0)
    return out.to(s.y.dtype), d_y.to(s.y.dtype), d_gates.to(s.gates.dtype)


def _plain_layer(s):
    a, a_scale = _quantised(_gathered(s.x.float(), s.order, s.topk))
    h = _plain_rows(a, a_scale, s.w1, s.w1_scale, s.offsets, s.cap).to(torch.bfloat16).float()
    b, b_scale = _quantised(_activate(h[:, : s.F], "silu") * h[:, s.F:])
    y = _plain_rows(b, b_scale, s.w2, s.w2_scale, s.offsets, s.cap).to(torch.bfloat16)
    return _joined(y, s.slot, s.gates).to(torch.bfloat16)


# ---- the definitions in 64 bits -------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return globals()["_exact_" + case["kind"]](s)


def _exact_activation(y, act):
    if act == "relu":
        return torch.relu(y)
    if act == "gelu":
        return y * torch.special.ndtr(y)
    if act == "silu":
        return y * torch.sigmoid(y)
    return y


def _exact_product(s):
    y = torch.mm(s.a.double(), s.b.double().t().contiguous())
    y *= torch.outer(s.a_scale.double(), s.b_scale.double())
    if s.c is not None:
        y += s.c.double()
    if s.bias_v is not None:
        y += s.bias_v.double()
    return _exact_activation(y, s.act)


def _exact_rows(a, a_scale, w, w_scale, offsets):
    y = torch.zeros(a.shape[0], w.shape[1], dtype=torch.float64, device="cuda")
    at = offsets.tolist()
    for e in range(len(at) - 1):
        r = slice(at[e], at[e + 1])
        if at[e + 1] > at[e]:
            y[r] = torch.mm(a[r].double(), w[e].double().t().contiguous())
            y[r] *= torch.outer(a_scale[r].double(), w_scale[e].double())
    return y


def _exact_experts(s):
    return _exact_activation(_exact_rows(s.a, s.a_scale, s.b, s.b_scale, s.offsets), s.act)


def _exact_codes(x):
    scale = (x.abs().amax(1) / INT8_MAX).clamp(min=MIN_SCALE)
    return torch.round(x / scale[:, None]).clamp(-INT8_MAX, INT8_MAX), scale


def _exact_gathered(x, index, div):
    y = torch.zeros(index.numel(), x.shape[1], dtype=torch.float64, device="cuda")
    live = index >= 0
    y[live] = x.double()[torch.div(index[live], div, rounding_mode="floor").long()]
    return y


def _exact_quant(s):
    q, scale = _exact_codes(s.x.double() if s.index is None else _exact_gathered(s.x, s.index, s.gather))
    return q.to(torch.int8), scale


def _exact_joined(y, slot, weights=None):
    out = torch.zeros(slot.shape[0], y.shape[1], dtype=torch.float64, device="cuda")
    for j in range(slot.shape[1]):
        live = slot[:, j] >= 0
        rows = y[slot[live, j].long()].double()
        out[live] += rows if weights is None else rows * weights[live, j].double()[:, None]
    return out


def _exact_sort(s):
    return _exact_gathered(s.x, s.order, s.topk), _exact_joined(s.d_y, s.slot)


def _exact_combine(s):
    d_y = _exact_gathered(s.d_out, s.order, s.topk)
    live = s.order >= 0
    d_y[live] *= s.gates.flatten()[s.order[live].long()].double()[:, None]
    d_gates = torch.zeros(s.tokens, s.topk, dtype=torch.float64, device="cuda")
    for j in range(s.topk):
        live = s.slot[:, j] >= 0
        d_gates[live, j] = (s.y[s.slot[live, j].long()].double() * s.d_out[live].double()).sum(1)
    return _exact_joined(s.y, s.slot, s.gates), d_y, d_gates


def _exact_layer(s):
    # what the layer keeps between its steps is rounded as its definition says: codes and bfloat16
    a, a_scale = _exact_codes(_exact_gathered(s.x, s.order, s.topk))
    h = _exact_rows(a, a_scale, s.w1, s.w1_scale, s.offsets).to(torch.bfloat16).double()
    b, b_scale = _exact_codes(_exact_activation(h[:, : s.F], "silu") * h[:, s.F:])
    y = _exact_rows(b, b_scale, s.w2, s.w2_scale, s.offsets).to(torch.bfloat16)
    return _exact_joined(y, s.slot, s.gates)
