"""The operators around an 8-bit expert layer, as cases to measure: products of e4m3 operands that
carry a scale for each block of 128, the quantisation that makes such operands, and the routing of
tokens to experts with its balance loss.

With `own` false, run() computes them from elementary torch operations; with `own` true it calls
the library's entry points (include/htscaled.h, include/htroute.h).
"""
import math
import types

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -126

# Sizes a draw stays within; the largest product is the benchmark's 8192^3.
MOST_FLOPS = 2 * 8192 ** 3


# ---- cases ---------------------------------------------------------------------------------

def listed():
    return [
        # one token through one linear layer: latency
        product("product 1x4096x4096", 1, 4096, 4096, bias=True),
        # a decode batch against a wide weight: the weight's bytes bound it
        product("product 16x16384x8192", 16, 16384, 8192),
        # a short prompt of an odd length, with a bias and an activation
        product("product 333x4096x8192", 333, 4096, 8192, bias=True, act="gelu"),
        # a training or prefill step
        product("product 8192x8192x8192", 8192, 8192, 8192),
        # the weight gradient of a linear layer: both operands scaled along the tokens, the result
        # added to a float32 gradient
        product("weight gradient 4096x8192x5008", 4096, 8192, 5008, out="f32", b_block=1, accumulate=True),
        # a decode step of an expert layer: few rows for each expert, all weights read
        experts("experts decode 128 rows of 64", 128, 64, 4096, 2048, act="silu"),
        # a prompt through an expert layer, weighted by the gates
        experts("experts prefill 8190 rows of 32", 8190, 32, 4096, 2048, gate=True),
        # the experts' weight gradients: each expert's own rows are summed over
        experts_grad("experts gradient 6000 rows of 16", 6000, 16, 2048, 2048),
        # one token's activations before a product
        quant("quantise 1x8192 bf16", 1, 8192, "bf16"),
        # a training step's activations, for the product and, transposed, for the weight gradient
        quant("quantise 8192x8192 bf16 both ways", 8192, 8192, "bf16", both=True),
        # a decode batch's routing, with its loss
        routing("route 37 tokens to 6 of 64", 37, 64, 6, 1, "bf16"),
        # a training batch's routing, groups aligned for the weight gradient
        routing("route 16384 tokens to 8 of 256", 16384, 256, 8, 128, "f32"),
    ]


def product(name, M, N, K, out="bf16", b_block=BLOCK, bias=False, act="none", accumulate=False):
    return {"name": name, "kind": "product", "M": M, "N": N, "K": K, "out": out, "b_block": b_block,
            "bias": bias, "act": act, "accumulate": accumulate}


def experts(name, rows, E, N, K, act="none", gate=False):
    return {"name": name, "kind": "experts", "rows": rows, "E": E, "N": N, "K": K, "act": act, "gate": gate}


def experts_grad(name, rows, E, M, N):
    return {"name": name, "kind": "experts_grad", "rows": rows, "E": E, "M": M, "N": N}


def quant(name, rows, cols, dtype, both=False, block_rows=1, pow2=False, gather=0):
    return {"name": name, "kind": "quant", "rows": rows, "cols": cols, "dtype": dtype, "both": both,
            "block_rows": block_rows, "pow2": pow2, "gather": gather}


def routing(name, tokens, E, topk, align, dtype):
    return {"name": name, "kind": "routing", "tokens": tokens, "E": E, "topk": topk, "align": align, "dtype": dtype}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["product", "product", "gradient", "experts", "experts", "experts_grad", "quant", "quant",
                       "weight", "routing", "routing"])
    if kind in ("product", "gradient"):
        while True:
            M, N, K = _log(rng, 1, 8192), _log(rng, 256, 16384), 16 * _log(rng, 8, 512)
            if 2 * M * N * K <= MOST_FLOPS:
                break
        if kind == "gradient":
            c = product("", max(M, 128), N, K, out="f32", b_block=1, accumulate=rng.random() < 0.5)
        else:
            c = product("", M, N, K, bias=rng.random() < 0.5, act=rng.choice(["none", "relu", "gelu", "silu"]))
    elif kind == "experts":
        while True:
            rows, E, N, K = _log(rng, 8, 16384), _log(rng, 4, 128), 8 * _log(rng, 32, 1024), 16 * _log(rng, 16, 512)
            if 2 * rows * N * K <= MOST_FLOPS / 4 and E * N * K <= 1 << 30:
                break
        c = experts("", rows, E, N, K, act=rng.choice(["none", "silu"]), gate=rng.random() < 0.5)
    elif kind == "experts_grad":
        while True:
            rows, E, M, N = _log(rng, 64, 16384), _log(rng, 4, 64), _log(rng, 256, 4096), _log(rng, 256, 4096)
            if 2 * rows * M * N <= MOST_FLOPS / 4 and E * M * N <= 1 << 28:
                break
        c = experts_grad("", rows, E, M, N)
    elif kind == "quant":
        rows, cols = _log(rng, 1, 16384), _log(rng, 128, 16384)
        if rows * cols > 1 << 26:
            rows = (1 << 26) // cols
        c = quant("", rows, cols, rng.choice(["bf16", "f16", "f32"]), both=rng.random() < 0.5,
                  pow2=rng.random() < 0.3, gather=rng.choice([0, 0, 2, 8]))
    elif kind == "weight":
        rows, cols = _log(rng, 256, 8192), _log(rng, 256, 8192)
        c = quant("", rows, cols, rng.choice(["bf16", "f32"]), both=rng.random() < 0.5, block_rows=BLOCK,
                  pow2=rng.random() < 0.3)
    else:
        E = _log(rng, 4, 512)
        c = routing("", _log(rng, 1, 32768), E, rng.randint(1, min(8, E)), rng.choice([1, 1, 16, 128]),
                    rng.choice(["f32", "bf16"]))
    del c["name"]
    return c


def _hit(rows, E):
    """Experts that at least one of `rows` evenly spread rows goes to."""
    return E * (1.0 - (1.0 - 1.0 / E) ** rows)


def _blocks(n):
    return -(-n // BLOCK)


def _up(n, m):
    return -(-n // m) * m


_SIZE = {"bf16": 2, "f16": 2, "f32": 4}
_TYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def work(case):
    kind = case["kind"]
    if kind == "product":
        M, N, K, kb = case["M"], case["N"], case["K"], _blocks(case["K"])
        size = _SIZE[case["out"]]
        b = M * K + N * K + 4 * kb * (M + -(-N // case["b_block"])) + M * N * size
        b += (N * size if case["bias"] else 0) + (M * N * size if case["accumulate"] else 0)
        return {"bytes": b, "flops": 2 * M * N * K}
    if kind == "experts":
        R, E, N, K, kb = case["rows"], case["E"], case["N"], case["K"], _blocks(case["K"])
        hit = _hit(R, E)
        b = R * K + hit * (N * K + 4 * kb * _blocks(N)) + 4 * kb * R + 2 * R * N + 4 * (E + 1)
        return {"bytes": int(b + (4 * R if case["gate"] else 0)), "flops": 2 * R * N * K}
    if kind == "experts_grad":
        R, E, M, N = case["rows"], case["E"], case["M"], case["N"]
        return {"bytes": R * (M + N) + 4 * _blocks(R) * (M + N) + 4 * E * M * N + 4 * (E + 1), "flops": 2 * R * M * N}
    if kind == "quant":
        n = case["rows"] * case["cols"]
        source = n // max(1, case["gather"]) * _SIZE[case["dtype"]]
        scales = 4 * (n // BLOCK if case["block_rows"] == 1 else n // BLOCK ** 2)
        return {"bytes": int(source + (n + scales) * (2 if case["both"] else 1)), "flops": 4 * n}
    T, E, k = case["tokens"], case["E"], case["topk"]
    rows = T * k + E * (case["align"] - 1)
    return {"bytes": 2 * T * E * _SIZE[case["dtype"]] + 4 * (2 * T * k + rows) + T + 16 * E, "flops": 16 * T * E}


# ---- inputs --------------------------------------------------------------------------------

def _split(x, dim, block):
    """x with zeros appended along `dim` to whole blocks, and that dimension as (blocks, block)."""
    n = x.shape[dim]
    pad = [0, 0] * (x.dim() - 1 - dim) + [0, _up(n, block) - n]
    return torch.nn.functional.pad(x, pad).unflatten(dim, (-1, block))


def _codes(x, scale, inverse):
    return (x * inverse).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _scales(amax, pow2):
    """The scale of blocks with the largest magnitudes `amax` and the factor the block's values are
    multiplied by; both in float32.  A block with a value that is not finite has scale NaN."""
    if pow2:
        # the least power of two that keeps amax / scale within the type's range
        e = torch.frexp((amax / E4M3_MAX).clamp(min=MIN_SCALE))
        exponent = torch.where(e.mantissa == 0.5, e.exponent - 1, e.exponent).clamp(-126, 127)
        scale = torch.ldexp(torch.ones_like(amax), exponent)
        inverse = torch.ldexp(torch.ones_like(amax), -exponent)
    else:
        top = amax.clamp(min=E4M3_MAX * MIN_SCALE)
        scale, inverse = top / E4M3_MAX, E4M3_MAX / top
    bad = ~torch.isfinite(amax)
    return scale.masked_fill(bad, math.nan), inverse.masked_fill(bad, math.nan)


def _rows_quantised(x, pow2=False):
    """e4m3 codes of x (..., rows, cols) and scales (..., rows, blocks), a scale for each 128 columns."""
    v = _split(x.float(), x.dim() - 1, BLOCK)
    scale, inverse = _scales(v.abs().amax(-1), pow2)
    return _codes(v, scale, inverse[..., None]).flatten(-2)[..., : x.shape[-1]], scale


def _blocks_quantised(x, pow2=False):
    """The same with a scale for each block of 128 rows and 128 columns."""
    d = x.dim()
    v = _split(_split(x.float(), d - 1, BLOCK), d - 2, BLOCK)   # (..., RB, 128, CB, 128)
    scale, inverse = _scales(v.abs().amax((-3, -1)), pow2)
    q = _codes(v, scale, inverse[..., :, None, :, None])
    return q.flatten(-2).flatten(-3, -2)[..., : x.shape[-2], : x.shape[-1]], scale


def _activations(g, rows, cols):
    """Normal values whose columns differ in size, a few by a lot."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    return x * torch.exp(0.7 * torch.randn(cols, generator=g, device="cuda"))


def _weights(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda") * shape[-1] ** -0.5


def _sizes(g, rows, E, align):
    """How many of `rows` rows each expert gets, and where the groups start, from one draw of an
    expert for each row, some experts preferred over others."""
    lean = torch.exp(0.5 * torch.randn(E, generator=g, device="cuda"))
    to = torch.multinomial(lean, rows, replacement=True, generator=g)
    sizes = torch.bincount(to, minlength=E).tolist()
    starts = [0]
    for n in sizes:
        starts.append(starts[-1] + _up(n, align))
    return sizes, starts


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


def _make(s, *sizes, **layout):
    from hierarchical_tiling_amd import htscaled
    s.gemm = htscaled.ScaledGemm(htscaled.make_desc(*sizes, **layout))
    s.workspace = torch.empty(s.gemm.workspace_bytes, dtype=torch.uint8, device="cuda")


def _prepare_product(s, g):
    a, a_scale = _rows_quantised(_activations(g, s.M, s.K))
    s.a, s.a_scale = a.contiguous(), a_scale.t().contiguous()           # scales (K blocks, M)
    if s.b_block == 1:
        b, b_scale = _rows_quantised(_activations(g, s.N, s.K))
        s.b_scale = b_scale.t().contiguous()                              # (K blocks, N)
    else:
        b, b_scale = _blocks_quantised(_weights(g, s.N, s.K))
        s.b_scale = b_scale.contiguous()                                  # (N blocks, K blocks)
    s.b = b.contiguous()
    s.out_type = _TYPE[s.out]
    s.bias_v = (0.1 * torch.randn(s.N, generator=g, device="cuda")).to(s.out_type) if s.bias else None
    s.c = torch.randn(s.M, s.N, generator=g, device="cuda").to(s.out_type) if s.accumulate else None
    s.d = torch.empty(s.M, s.N, dtype=s.out_type, device="cuda")


def _plan_product(s):
    _make(s, s.M, s.N, s.K, s.out, lda=s.K, ldb=s.K, ldd=s.N, ldc=s.N if s.accumulate else 0, b_block=s.b_block,
          a_scale_strides=(1, s.M), b_scale_strides=(1, s.N) if s.b_block == 1 else (_blocks(s.K), 1),
          bias=s.bias, act=s.act)


def _prepare_experts(s, g):
    sizes, starts = _sizes(g, s.rows, s.E, 1)
    s.cap = max(sizes)
    s.offsets = torch.tensor(starts, dtype=torch.int32, device="cuda")
    a, a_scale = _rows_quantised(_activations(g, s.rows, s.K))
    s.a, s.a_scale = a.contiguous(), a_scale.t().contiguous()
    b, b_scale = _blocks_quantised(_weights(g, s.E, s.N, s.K))
    s.b, s.b_scale = b.contiguous(), b_scale.contiguous()                # (E, N blocks, K blocks)
    s.gates = torch.rand(s.rows, generator=g, device="cuda") if s.gate else None
    s.d = torch.empty(s.rows, s.N, dtype=torch.bfloat16, device="cuda")


def _plan_experts(s):
    nb, kb = _blocks(s.N), _blocks(s.K)
    _make(s, s.rows, s.N, s.K, "bf16", lda=s.K, ldb=s.K, ldd=s.N, a_scale_strides=(1, s.rows),
          b_scale_strides=(kb, 1), act=s.act, row_scale=s.gate, groups="rows", batch=s.E, b_stride_l=s.N * s.K,
          b_scale_l=nb * kb)


def _prepare_experts_grad(s, g):
    # each expert's rows start on a multiple of 128 and are filled up to one with zeros
    sizes, starts = _sizes(g, s.rows, s.E, BLOCK)
    s.cap = max(_up(n, BLOCK) for n in sizes)
    s.total = max(starts[-1], BLOCK)
    s.offsets = torch.tensor(starts, dtype=torch.int32, device="cuda")
    live = torch.zeros(s.total, device="cuda")
    for e, n in enumerate(sizes):
        live[starts[e]: starts[e] + n] = 1
    a, a_scale = _rows_quantised(_activations(g, s.total, s.M).t() * live)
    b, b_scale = _rows_quantised(_activations(g, s.total, s.N).t() * live)
    s.a, s.a_scale = a.contiguous(), a_scale.t().contiguous()            # (M, total), (total blocks, M)
    s.b, s.b_scale = b.contiguous(), b_scale.t().contiguous()
    s.d = torch.empty(s.E, s.M, s.N, device="cuda")


def _plan_experts_grad(s):
    _make(s, s.M, s.N, s.total, "f32", lda=s.total, ldb=s.total, ldd=s.N, b_block=1, a_scale_strides=(1, s.M),
          b_scale_strides=(1, s.N), groups="k", batch=s.E, d_stride_l=s.M * s.N)


def _prepare_quant(s, g):
    # gather > 0: each source row goes to about `gather` rows of the result, in a shuffled order
    # with a few empty places, as tokens go to their experts' rows
    source = max(1, s.rows // max(1, s.gather))
    s.x = _activations(g, source, s.cols).to(_TYPE[s.dtype])
    s.index = None
    if s.gather:
        s.index = torch.randint(-s.gather, source * s.gather, (s.rows,), generator=g, device="cuda", dtype=torch.int32)
    pitch, pitch_t = _up(s.cols, 16), _up(s.rows, 16)
    s.q = torch.zeros(s.rows, pitch, dtype=torch.float8_e4m3fn, device="cuda")[:, : s.cols]
    s.qt = torch.zeros(s.cols, pitch_t, dtype=torch.float8_e4m3fn, device="cuda")[:, : s.rows] if s.both else None
    rb, cb = _blocks(s.rows), _blocks(s.cols)
    if s.block_rows == 1:
        s.scale = torch.empty(cb, s.rows, device="cuda").t()             # (rows, column blocks)
        s.scale_t = torch.empty(rb, s.cols, device="cuda").t() if s.both else None
    else:
        s.scale, s.scale_t = torch.empty(rb, cb, device="cuda"), None


def _prepare_routing(s, g):
    lean = 0.7 * torch.randn(s.E, generator=g, device="cuda")
    s.logits = (torch.randn(s.tokens, s.E, generator=g, device="cuda") + lean).to(_TYPE[s.dtype])
    s.ids = s.logits.float().topk(s.topk, dim=1).indices.to(torch.int32).contiguous()
    # the last sixteenth of the tokens is padding
    s.mask = (torch.arange(s.tokens, device="cuda") < s.tokens - s.tokens // 16).to(torch.uint8)
    s.coef = 0.01
    s.d_loss = 0.5 + torch.rand(1, generator=g, device="cuda")
    s.places = s.tokens * s.topk + s.E * (s.align - 1)
    i32 = dict(dtype=torch.int32, device="cuda")
    s.counts, s.offsets = torch.empty(s.E, **i32), torch.empty(s.E + 1, **i32)
    s.order, s.slot = torch.empty(s.places, **i32), torch.empty(s.tokens, s.topk, **i32)
    s.loss, s.prob, s.live = torch.empty(1, device="cuda"), torch.empty(s.E, device="cuda"), torch.empty(1, **i32)
    s.d_logits = torch.empty_like(s.logits)


def _plan_routing(s):
    from hierarchical_tiling_amd import htroute
    s.workspace = torch.empty(htroute.workspace_size(s.tokens, s.topk, s.E), dtype=torch.uint8, device="cuda")


# ---- one pass ------------------------------------------------------------------------------

def run(s):
    return globals()[("_own_" if own else "_plain_") + s.kind](s)


def _own_product(s):
    s.gemm.run(s.a, s.a_scale, s.b, s.b_scale, s.d, C=s.c, bias=s.bias_v, beta=1.0 if s.accumulate else 0.0,
               workspace=s.workspace)
    return s.d


def _own_experts(s):
    s.gemm.run(s.a, s.a_scale, s.b, s.b_scale, s.d, row_scale=s.gates, offsets=s.offsets, workspace=s.workspace)
    return s.d


def _own_experts_grad(s):
    s.gemm.run(s.a, s.a_scale, s.b, s.b_scale, s.d, offsets=s.offsets, workspace=s.workspace)
    return s.d


def _own_quant(s):
    from hierarchical_tiling_amd import htscaled
    htscaled.quantize(s.x, s.q, s.scale, s.qt, s.scale_t, block_rows=s.block_rows, pow2=s.pow2, row_index=s.index,
                      index_div=max(1, s.gather))
    return [t for t in (s.q, s.scale, s.qt, s.scale_t) if t is not None]


def _own_routing(s):
    from hierarchical_tiling_amd import htroute
    htroute.route(s.ids, s.counts, s.offsets, s.order, s.slot, mask=s.mask, align=s.align, workspace=s.workspace)
    htroute.balance_loss(s.logits, s.counts, s.topk, s.loss, s.prob, s.live, mask=s.mask, coef=s.coef,
                         workspace=s.workspace)
    htroute.balance_grad(s.logits, s.counts, s.topk, s.live, s.d_loss, s.d_logits, mask=s.mask, coef=s.coef)
    return s.counts, s.offsets, s.order, s.slot, s.loss, s.prob, s.d_logits


def _activate(y, act):
    if act == "relu":
        return y.clamp(min=0)
    if act == "gelu":
        return 0.5 * y * (1 + torch.erf(y * 0.5 ** 0.5))
    if act == "silu":
        return y / (1 + torch.exp(-y))
    return y


def _values(q, scale):
    """The float32 values of codes q (..., rows, cols) with scales (..., rows, blocks of 128 columns)."""
    return q.float() * scale.repeat_interleave(BLOCK, -1)[..., : q.shape[-1]]


def _weight_values(q, scale):
    """The same with a scale for each block of 128 rows and columns."""
    return _values(q, scale.repeat_interleave(BLOCK, -2)[..., : q.shape[-2], :])


def _plain_product(s):
    a = _values(s.a, s.a_scale.t())
    b = _values(s.b, s.b_scale.t()) if s.b_block == 1 else _weight_values(s.b, s.b_scale)
    y = a @ b.t()
    if s.c is not None:
        y = y + s.c.float()
    if s.bias_v is not None:
        y = y + s.bias_v.float()
    return _activate(y, s.act).to(s.out_type)


def _places(s, rows):
    """Rows in groups to a place of their own in (E, cap): group and index within it."""
    row = torch.arange(rows, device="cuda")
    group = (row[:, None] >= s.offsets[None, 1:]).sum(1).clamp(max=s.E - 1)
    return group, row - s.offsets[group]


def _plain_experts(s):
    group, at = _places(s, s.rows)
    x = torch.zeros(s.E, s.cap, s.K, device="cuda")
    x[group, at] = _values(s.a, s.a_scale.t())
    w = _weight_values(s.b, s.b_scale).transpose(1, 2).contiguous()
    y = torch.bmm(x, w)[group, at]
    if s.gates is not None:
        y = y * s.gates[:, None]
    return _activate(y, s.act).to(torch.bfloat16)


def _plain_experts_grad(s):
    group, at = _places(s, s.total)
    a = torch.zeros(s.E, s.cap, s.M, device="cuda")
    b = torch.zeros(s.E, s.cap, s.N, device="cuda")
    a[group, at] = _values(s.a, s.a_scale.t()).t()
    b[group, at] = _values(s.b, s.b_scale.t()).t()
    return torch.bmm(a.transpose(1, 2).contiguous(), b)


def _plain_quant(s):
    x = s.x.float()
    if s.index is not None:
        # an index below zero leaves a row of zeros
        x = x[(s.index.clamp(min=0) // s.gather).long()] * (s.index >= 0)[:, None]
    if s.block_rows == BLOCK:
        q, scale = _blocks_quantised(x, s.pow2)
        return [q, scale] + ([q.t().contiguous()] if s.both else [])
    q, scale = _rows_quantised(x, s.pow2)
    if not s.both:
        return [q, scale]
    qt, scale_t = _rows_quantised(x.t(), s.pow2)
    return [q, scale, qt, scale_t]


def _plain_routing(s):
    T, E, k = s.tokens, s.E, s.topk
    live = s.mask.bool()
    valid = live[:, None] & (s.ids >= 0) & (s.ids < E)
    flat = torch.where(valid, s.ids, E).flatten().long()
    counts = torch.zeros(E + 1, dtype=torch.int32, device="cuda").index_add_(
        0, flat, torch.ones_like(flat, dtype=torch.int32))
    starts = torch.cumsum(counts, 0) - counts
    groups = (counts[:E] + s.align - 1) // s.align * s.align
    offsets = torch.cat([torch.zeros_like(groups[:1]), torch.cumsum(groups, 0)]).int()
    by_expert = torch.argsort(flat, stable=True)
    to = flat[by_expert]
    place = torch.arange(T * k, device="cuda") - starts[to] + offsets[to]
    place = torch.where(to < E, place, -1)
    slot = torch.empty(T * k, dtype=torch.int32, device="cuda")
    slot[by_expert] = place.int()
    order = torch.full((s.places + 1,), -1, dtype=torch.int32, device="cuda")
    order[place] = by_expert.int()          # place -1 is the extra last entry
    # the balance loss: coef * E * sum over e of (share of the assignments) * (mean probability)
    x = s.logits.float()
    p = torch.exp(x - x.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True) * live[:, None]
    n = live.sum().clamp(min=1)
    prob = (p.sum(0, dtype=torch.float64) / n).float()
    share = counts[:E].float() * E / (k * n)
    loss = s.coef * (share.double() * prob.double()).sum().float().reshape(1)
    pull = s.d_loss * s.coef * (share - 1) / n           # a constant added to all drops out
    d_logits = p * (pull - (p * pull).sum(1, keepdim=True))
    return counts[:E], offsets, order[: s.places], slot.view(T, k), loss, prob, d_logits.to(s.logits.dtype)


# ---- the definitions in 64 bits -------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return globals()["_exact_" + case["kind"]](s)


def _wide(q, scale, row_block, col_block):
    """Codes times scales, element by element, in float64: scale[r // row_block, c // col_block]."""
    r = torch.arange(q.shape[0], device=q.device) // row_block
    c = torch.arange(q.shape[1], device=q.device) // col_block
    return q.double() * scale.double()[r][:, c]


def _exact_activation(y, act):
    if act == "relu":
        return torch.relu(y)
    if act == "gelu":
        return y * torch.special.ndtr(y)
    if act == "silu":
        return y * torch.sigmoid(y)
    return y


def _exact_product(s):
    a = _wide(s.a, s.a_scale.t(), 1, BLOCK)
    b = _wide(s.b, s.b_scale.t(), 1, BLOCK) if s.b_block == 1 else _wide(s.b, s.b_scale, BLOCK, BLOCK)
    y = torch.mm(a, b.t().contiguous())
    if s.c is not None:
        y += s.c.double()
    if s.bias_v is not None:
        y += s.bias_v.double()
    return _exact_activation(y, s.act)


def _exact_experts(s):
    a = _wide(s.a, s.a_scale.t(), 1, BLOCK)
    y = torch.zeros(s.rows, s.N, dtype=torch.float64, device="cuda")
    at = s.offsets.tolist()
    for e in range(s.E):
        if at[e + 1] > at[e]:
            w = _wide(s.b[e], s.b_scale[e], BLOCK, BLOCK)
            y[at[e]: at[e + 1]] = torch.mm(a[at[e]: at[e + 1]], w.t().contiguous())
    if s.gates is not None:
        y *= s.gates.double()[:, None]
    return _exact_activation(y, s.act)


def _exact_experts_grad(s):
    a, b = _wide(s.a, s.a_scale.t(), 1, BLOCK), _wide(s.b, s.b_scale.t(), 1, BLOCK)
    y = torch.zeros(s.E, s.M, s.N, dtype=torch.float64, device="cuda")
    at = s.offsets.tolist()
    for e in range(s.E):
        if at[e + 1] > at[e]:
            y[e] = torch.mm(a[:, at[e]: at[e + 1]].contiguous(), b[:, at[e]: at[e + 1]].t().contiguous())
    return y


def _nearest_e4m3(v):
    """The nearest e4m3 value (3 bits after the point, least exponent -6, ties to even), saturating."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -40))).clamp(min=-6)
    quantum = torch.exp2(e - 3)
    return (torch.round(v / quantum) * quantum).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_blocks(x, row_block, col_block, pow2):
    """Codes' values and scales of float64 x, a scale for each row_block x col_block."""
    rows, cols = x.shape
    rb, cb = -(-rows // row_block), -(-cols // col_block)
    top = torch.zeros(rb, cols, dtype=torch.float64, device=x.device)
    r = torch.arange(rows, device=x.device) // row_block
    top.index_reduce_(0, r, x.abs(), "amax")
    amax = torch.zeros(rb, cb, dtype=torch.float64, device=x.device)
    c = torch.arange(cols, device=x.device) // col_block
    amax.index_reduce_(1, c, top, "amax")
    scale = (amax / E4M3_MAX).clamp(min=MIN_SCALE)
    if pow2:
        scale = torch.exp2(torch.ceil(torch.log2(scale)))
    return _nearest_e4m3(x / scale[r][:, c]), scale


def _exact_quant(s):
    x = s.x.double()
    if s.index is not None:
        gathered = torch.zeros(s.rows, s.cols, dtype=torch.float64, device="cuda")
        live = s.index >= 0
        gathered[live] = x[torch.div(s.index[live], s.gather, rounding_mode="floor").long()]
        x = gathered
    q, scale = _exact_blocks(x, s.block_rows, BLOCK, s.pow2)
    if not s.both:
        return [q, scale]
    if s.block_rows == BLOCK:
        return [q, scale, q.t().contiguous()]
    qt, scale_t = _exact_blocks(x.t().contiguous(), 1, BLOCK, s.pow2)
    return [q, scale, qt, scale_t]


def _exact_routing(s):
    ids, live = s.ids.cpu(), s.mask.cpu().bool()
    T, k = ids.shape
    groups = [[] for _ in range(s.E)]
    for i, e in enumerate(ids.flatten().tolist()):
        if live[i // k] and 0 <= e < s.E:
            groups[e].append(i)
    counts = torch.tensor([len(v) for v in groups], dtype=torch.int32)
    offsets, order = [0], torch.full((s.places,), -1, dtype=torch.int32)
    slot = torch.full((T * k,), -1, dtype=torch.int32)
    for members in groups:
        at = offsets[-1]
        for j, i in enumerate(members):
            order[at + j] = i
            slot[i] = at + j
        offsets.append(at + _up(len(members), s.align))
    p = torch.softmax(s.logits.double(), 1) * s.mask.double()[:, None]
    n = max(1, int(live.sum()))
    f = counts.double().cuda() * s.E / (k * n)
    prob = p.sum(0) / n
    loss = (s.coef * (f * prob).sum()).reshape(1)
    g = s.d_loss.double() * s.coef * f / n
    d_logits = p * (g - torch.mv(p, g)[:, None])
    d_logits *= s.mask.double()[:, None]
    return counts, torch.tensor(offsets, dtype=torch.int32), order, slot.view(T, k), loss, prob, d_logits
