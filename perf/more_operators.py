"""What is timed of the operators around and inside a mixture-of-experts block.

Three operators beside the ragged products, the router and the join:

  gated  the gated feed-forward block of experts with any number of rows: gate and
         up projection with the activation and the product in one kernel, and the
         backward pass of the activation inside the down projection's gradient
  fp8    tokens and weights quantized to 8-bit floating point (e4m3) with a scale for
         each block of 128, and their product grouped by expert
  norm   what follows a block: its output normalized, gated and added to the scaled
         residual, and the sum normalized for the next block; and the gradients

`own` chooses between the plain torch form of each and the package's calls.
"""

import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "fp16": 2, "f32": 4}
_EPS = 1e-6

# What a drawn case may cost at most: the largest listed product, weights that leave room
# for several sets of inputs, the largest listed norm.
_FLOPS = 2 * 16384 * 4096 * 14336
_WEIGHTS = 1 << 29
_NORM = 16384 * 4096


def _gated(name, dtype, experts, active, tokens, top_k, hidden, ffn, keep_h):
    """The forward pass: tokens * top_k rows; `active` experts have rows, the others none.
    keep_h: both projections are kept for the backward pass."""
    return {"name": name, "op": "gated", "dtype": dtype, "experts": experts, "active": active,
            "tokens": tokens, "top_k": top_k, "hidden": hidden, "ffn": ffn, "keep_h": keep_h}


def _gated_bwd(name, dtype, experts, active, tokens, top_k, hidden, ffn):
    return {"name": name, "op": "gated_bwd", "dtype": dtype, "experts": experts, "active": active,
            "tokens": tokens, "top_k": top_k, "hidden": hidden, "ffn": ffn}


def _fp8(name, dtype, out, experts, active, tokens, top_k, k, n):
    return {"name": name, "op": "fp8", "dtype": dtype, "out": out, "experts": experts,
            "active": active, "tokens": tokens, "top_k": top_k, "k": k, "n": n}


def _fp8_weights(name, dtype, experts, n, k):
    return {"name": name, "op": "fp8_weights", "dtype": dtype, "experts": experts, "n": n, "k": k}


def _norm(name, dtype, residual, tokens, hidden, post, gate, backward):
    """post: the block's output is normalized before it is added; gate: a factor for each
    token; residual: the type of the residual stream."""
    return {"name": name, "op": "norm", "dtype": dtype, "residual": residual, "tokens": tokens,
            "hidden": hidden, "post": post, "gate": gate, "backward": backward}


def listed():
    return [
        # training of an 8-expert layer (hidden 4096, FFN 14336): 4096 tokens, two experts each
        _gated("gated forward 8x4096x14336", "bf16", 8, 8, 4096, 2, 4096, 14336, True),
        # a prompt batch over many experts under skewed routing, 38 of 128 with no token
        _gated("gated forward 128x7168x1024", "fp16", 128, 90, 4096, 8, 7168, 1024, False),
        # nothing is a multiple of anything: a small odd model in training
        _gated("gated forward odd 5x1031x517", "fp16", 5, 4, 1777, 1, 1031, 517, True),
        # decoding 8 sequences: a row or two for each expert
        _gated("gated decode 8x4096x14336", "bf16", 8, 7, 8, 2, 4096, 14336, False),
        # the backward pass of the first: gradient of both projections, the activation anew
        _gated_bwd("gated backward 8x4096x14336", "bf16", 8, 8, 4096, 2, 4096, 14336),
        # serving in 8-bit floating point: a prompt batch
        _fp8("fp8 prompt 8x4096x14336", "bf16", "bf16", 8, 8, 8192, 2, 4096, 14336),
        # 8 sequences decoded over many experts, eight for each token
        _fp8("fp8 decode 128x7168x2048", "bf16", "bf16", 128, 48, 8, 8, 7168, 2048),
        # blocks of 128 that end inside the sizes, fp32 results
        _fp8("fp8 odd 3x1000x4099", "fp16", "f32", 3, 3, 333, 1, 1000, 4099),
        # the weights of a layer laid out for it
        _fp8_weights("fp8 weights 8x14336x4096", "bf16", 8, 14336, 4096),
        # after a block in a training step, and its gradients
        _norm("norm step 16384x4096", "bf16", "bf16", 16384, 4096, True, True, True),
        # an odd width, the residual stream in fp32
        _norm("norm step 1777x1031", "fp16", "f32", 1777, 1031, True, False, True),
        # a handful of decoded tokens: latency
        _norm("norm 5x7168", "bf16", "bf16", 5, 7168, False, False, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A feature count: mostly a multiple of 8, one in four any number."""
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.25 else max(8, v // 8 * 8)


def _sizes(rng, wide=1):
    """Rows and weights of a drawn product within what the largest listed one costs; its
    weights have wide * n rows."""
    k, n = _width(rng, 128, 8192), _width(rng, 128, 14336)
    experts = _log(rng, 1, max(1, min(256, _WEIGHTS // (wide * k * n))))
    top_k = min(experts, rng.choice([1, 1, 2, 4, 8]))
    most = max(1, int(_FLOPS / (2.0 * wide * k * n * top_k)))
    tokens = _log(rng, 1, max(1, min(32768 // top_k, most)))
    active = rng.randint(max(1, min(experts, tokens * top_k) // 2), min(experts, tokens * top_k))
    return experts, active, tokens, top_k, k, n


def draw(rng):
    kind = rng.choice(["gated", "gated", "gated_bwd", "fp8", "fp8", "fp8_weights", "norm", "norm"])
    if kind == "gated":
        case = _gated("", rng.choice(["bf16", "fp16"]), *_sizes(rng, 2), rng.random() < 0.5)
    elif kind == "gated_bwd":
        case = _gated_bwd("", rng.choice(["bf16", "fp16"]), *_sizes(rng, 2))
    elif kind == "fp8":
        case = _fp8("", rng.choice(["bf16", "fp16"]), rng.choice(["bf16", "bf16", "fp16", "f32"]),
                    *_sizes(rng))
    elif kind == "fp8_weights":
        n, k = _width(rng, 64, 14336), _width(rng, 64, 14336)
        case = _fp8_weights("", rng.choice(["bf16", "fp16"]),
                            _log(rng, 1, max(1, min(256, _WEIGHTS // (n * k)))), n, k)
    else:
        hidden = _width(rng, 64, 16384)
        dtype = rng.choice(["bf16", "fp16"])
        case = _norm("", dtype, rng.choice([dtype, "f32"]), _log(rng, 1, _NORM // hidden), hidden,
                     rng.random() < 0.7, rng.random() < 0.5, rng.random() < 0.6)
    del case["name"]
    return case


def _splits(case, gen):
    """Rows of each expert: `active` of them, chosen at random, with shares that
    differ by a log-normal factor; each has one row at least."""
    rows, experts, active = case["tokens"] * case["top_k"], case["experts"], case["active"]
    live = torch.randperm(experts, generator=gen)[:active]
    share = torch.randn(active, generator=gen).mul(0.8).exp()
    extra = torch.multinomial(share, rows - active, replacement=True, generator=gen) \
        if rows > active else torch.zeros(0, dtype=torch.int64)
    counts = torch.zeros(experts, dtype=torch.int64)
    counts[live] = 1 + torch.bincount(extra, minlength=active)
    return counts


def _rows(case, seed):
    """The routing of a product: splits on the host and the device, and the token of each row
    (every token in top_k rows, ascending within each expert)."""
    gen = torch.Generator().manual_seed(seed)
    counts = _splits(case, gen)
    rows, tokens = case["tokens"] * case["top_k"], case["tokens"]
    token = torch.randperm(tokens, generator=gen).repeat(case["top_k"])
    expert = torch.repeat_interleave(torch.arange(case["experts"]), counts)
    order = torch.argsort(expert * tokens + token)
    return {"splits": counts.tolist(), "m_splits": counts.cuda(), "rows": rows,
            "row_index": token[order].to(torch.int32).cuda()}


def _normal(shape, seed, dtype, std=1.0):
    gen = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").mul_(std).to(dtype)


def _uniform(shape, seed, lo, hi):
    gen = torch.Generator("cuda").manual_seed(seed)
    return torch.rand(shape, generator=gen, device="cuda") * (hi - lo) + lo


def prepare(case, seed):
    dtype = _TYPES[case["dtype"]]
    state = {"case": case}
    if case["op"] == "gated":
        state |= _rows(case, seed)
        g, h, f = case["experts"], case["hidden"], case["ffn"]
        state["x"] = _normal((case["tokens"], h), seed + 1, dtype)
        state["w"] = _normal((g, 2 * f, h), seed + 2, dtype, h ** -0.5)   # gate | up
    elif case["op"] == "gated_bwd":
        state |= _rows(case, seed)
        g, h, f = case["experts"], case["hidden"], case["ffn"]
        state["dy"] = _normal((state["rows"], h), seed + 1, dtype)
        state["w"] = _normal((g, h, f), seed + 2, dtype, f ** -0.5)       # down projection
        state["h"] = _normal((state["rows"], 2 * f), seed + 3, dtype)
    elif case["op"] == "fp8":
        state |= _rows(case, seed)
        g, k, n = case["experts"], case["k"], case["n"]
        state["x"] = _normal((case["tokens"], k), seed + 1, dtype)
        # codes of normal weights whose largest of a block is near 448
        gen = torch.Generator("cuda").manual_seed(seed + 2)
        state["wq"] = torch.randn((g, n, k), generator=gen, device="cuda").mul_(110.0) \
            .clamp_(-448, 448).to(torch.float8_e4m3fn)
        state["ws"] = _uniform((g, -(-n // 128), -(-k // 128)), seed + 3, 1e-4, 3e-4)
    elif case["op"] == "fp8_weights":
        g, n, k = case["experts"], case["n"], case["k"]
        state["w"] = _normal((g, n, k), seed + 1, dtype, 0.02)
    else:
        t, h = case["tokens"], case["hidden"]
        res = _TYPES[case["residual"]]
        # a residual stream grows, a few of its channels far above the rest
        loud = torch.where(_uniform((h,), seed + 6, 0, 1) < 0.01, 20.0, 1.0)
        state["x"] = (_normal((t, h), seed + 1, torch.float32, 2.0) * loud).to(res)
        state["f"] = _normal((t, h), seed + 2, dtype, 0.7)
        state["pre"] = _uniform((h,), seed + 3, 0.5, 1.5)
        state["post"] = _uniform((h,), seed + 4, 0.1, 0.6) if case["post"] else None
        state["gate"] = _uniform((t,), seed + 5, 0, 1) if case["gate"] else None
        state["scale"] = 0.875
        if case["backward"]:
            state["dy"] = _normal((t, h), seed + 7, dtype)
            state["dr"] = _normal((t, h), seed + 8, res)
    return state


# ----------------------------------------------------------------------------
# the plain forms
# ----------------------------------------------------------------------------

def _sigmoid(g):
    return 1.0 / (1.0 + torch.exp(-g))


def _plain_gated(state):
    x = state["x"][state["row_index"].long()]
    parts = zip(x.split(state["splits"]), state["w"])
    h = torch.cat([a.float() @ w.float().t() for a, w in parts])
    gate, up = h.chunk(2, dim=1)
    got = {"a": (gate * _sigmoid(gate) * up).to(x.dtype)}
    if state["case"]["keep_h"]:
        got["h"] = h.to(x.dtype)
    return got


def _plain_gated_bwd(state):
    parts = zip(state["dy"].split(state["splits"]), state["w"])
    da = torch.cat([dy.float() @ w.float() for dy, w in parts])
    gate, up = state["h"].float().chunk(2, dim=1)
    s = _sigmoid(gate)
    dh = torch.cat([da * up * s * (1.0 + gate * (1.0 - s)), da * gate * s], 1)
    return {"dh": dh.to(state["dy"].dtype), "a": (gate * s * up).to(state["dy"].dtype)}


def _e4m3(v):
    """The nearest of the e4m3 values, ties to the even one, of 64-bit values up to 448 (and
    what lies above by a rounding)."""
    exponent = torch.frexp(v).exponent - 1            # 2^exponent <= |v|
    step = torch.exp2((exponent.clamp(min=-6) - 3).double())
    return (torch.round(v / step) * step).clamp(-448, 448)


def _blocks_of(amax, shape, dims):
    """Maxima or scales of blocks of 128 spread over their values."""
    for d in dims:
        amax = amax.repeat_interleave(128, dim=d).narrow(d, 0, shape[d])
    return amax


def _plain_quantize(x):
    """Codes (as 64-bit values) and scales of each row's blocks of 128."""
    t, k = x.shape
    wide = torch.nn.functional.pad(x.abs(), (0, -k % 128)).view(t, -1, 128)
    # the stored scale is the fp32 value nearest to amax / 448, and a quotient next to the
    # border between two codes is decided in 64 bits
    scale = (wide.amax(2).double() / 448).float()
    over = _blocks_of(scale, x.shape, (1,)).double()
    return _e4m3(torch.where(over > 0, x.double() / over, 0.0)), scale


def _plain_fp8(state):
    q, scale = _plain_quantize(state["x"])
    x = q.float() * _blocks_of(scale, q.shape, (1,))
    shape = state["wq"].shape[1:]
    parts = zip(x[state["row_index"].long()].split(state["splits"]), state["wq"], state["ws"])
    return torch.cat([a @ (w.float() * _blocks_of(s, shape, (0, 1))).t() for a, w, s in parts]) \
        .to(_TYPES[state["case"]["out"]])


def _plain_fp8_weights(state):
    w = state["w"]
    g, n, k = w.shape
    wide = torch.nn.functional.pad(w.abs(), (0, -k % 128, 0, -n % 128))
    scale = (wide.view(g, -(-n // 128), 128, -(-k // 128), 128).amax((2, 4)).double() / 448).float()
    over = _blocks_of(scale, w.shape, (1, 2)).double()
    return {"q": _e4m3(torch.where(over > 0, w.double() / over, 0.0)).to(torch.float8_e4m3fn),
            "scale": scale}


def _normalized(v):
    return v * torch.rsqrt((v * v).mean(1, keepdim=True) + _EPS)


def _norm_grad(dn, v):
    """Gradient of v from that of _normalized(v)."""
    rs = torch.rsqrt((v * v).mean(1, keepdim=True) + _EPS)
    n = v * rs
    return rs * (dn - n * (dn * n).mean(1, keepdim=True))


def _plain_norm(state):
    case, f, gate = state["case"], state["f"].float(), state["gate"]
    b = _normalized(f) * state["post"] if case["post"] else f
    add = b * gate[:, None] if case["gate"] else b
    # the next norm is of the residual stream as it is stored
    r = (state["scale"] * state["x"].float() + add).to(state["x"].dtype)
    rf = r.float()
    got = {"r": r, "y": (_normalized(rf) * state["pre"]).to(state["f"].dtype)}
    if case["backward"]:
        dy = state["dy"].float()
        total = state["dr"].float() + _norm_grad(dy * state["pre"], rf)
        db = total * gate[:, None] if case["gate"] else total
        got["dx"] = (state["scale"] * total).to(r.dtype)
        got["dpre"] = (dy * _normalized(rf)).sum(0)
        if case["post"]:
            got["dpost"] = (db * _normalized(f)).sum(0)
            db = _norm_grad(db * state["post"], f)
        got["df"] = db.to(state["f"].dtype)
        if case["gate"]:
            got["dgate"] = (total * b).sum(1)
    return got


# ----------------------------------------------------------------------------
# the package's calls
# ----------------------------------------------------------------------------

def _own(state):
    import moe_expert_grouped_group_amd as mx
    case = state["case"]
    if case["op"] == "gated":
        h, a = mx.ragged_gemm_swiglu(state["x"], state["w"], state["m_splits"],
                                     row_index=state["row_index"], want_h=case["keep_h"])
        return {"a": a, "h": h} if case["keep_h"] else {"a": a}
    if case["op"] == "gated_bwd":
        dh, a = mx.ragged_gemm_swiglu_bwd(state["dy"], state["w"], state["h"], state["m_splits"])
        return {"dh": dh, "a": a}
    if case["op"] == "fp8":
        q, scale = mx.quantize_fp8(state["x"])
        return mx.ragged_gemm_fp8(q, scale, state["wq"], state["ws"], state["m_splits"],
                                  row_index=state["row_index"], out_dtype=_TYPES[case["out"]])
    if case["op"] == "fp8_weights":
        q, scale = mx.quantize_fp8_weight(state["w"])
        return {"q": q, "scale": scale}
    around = dict(residual_scale=state["scale"], gate=state["gate"], post_weight=state["post"],
                  pre_weight=state["pre"], eps=_EPS)
    r, y = mx.residual_norm(state["x"], state["f"], **around)
    got = {"r": r, "y": y}
    if case["backward"]:
        grad = mx.residual_norm_bwd(state["dy"], state["dr"], r, state["f"], **around)
        got |= {"dx": grad.x, "df": grad.f, "dpre": grad.pre_weight}
        if case["post"]:
            got["dpost"] = grad.post_weight
        if case["gate"]:
            got["dgate"] = grad.gate
    return got


def run(state):
    if own:
        return _own(state)
    return {"gated": _plain_gated, "gated_bwd": _plain_gated_bwd, "fp8": _plain_fp8,
            "fp8_weights": _plain_fp8_weights, "norm": _plain_norm}[state["case"]["op"]](state)


def work(case):
    """Each input read once, each output written once; the weights of experts
    without rows are not read."""
    e = _SIZE[case["dtype"]]
    if case["op"] in ("gated", "gated_bwd"):
        t, r, h, f = case["tokens"], case["tokens"] * case["top_k"], case["hidden"], case["ffn"]
        side = 8 * case["experts"]
        if case["op"] == "gated":
            moved = t * h + 2 * case["active"] * f * h + r * f * (3 if case["keep_h"] else 1)
            return {"bytes": moved * e + 4 * r + side, "flops": 4.0 * r * h * f}
        moved = r * h + case["active"] * f * h + r * f * 5
        return {"bytes": moved * e + side, "flops": 2.0 * r * h * f}
    if case["op"] == "fp8":
        t, r, k, n = case["tokens"], case["tokens"] * case["top_k"], case["k"], case["n"]
        moved = t * k * e + case["active"] * (n * k + 4 * -(-n // 128) * -(-k // 128))
        moved += r * n * _SIZE[case["out"]] + 4 * r + 8 * case["experts"]
        return {"bytes": moved, "flops": 2.0 * r * k * n}
    if case["op"] == "fp8_weights":
        g, n, k = case["experts"], case["n"], case["k"]
        return {"bytes": g * (n * k * (e + 1) + 4 * -(-n // 128) * -(-k // 128)),
                "flops": 2.0 * g * n * k}
    t, h, s = case["tokens"], case["hidden"], _SIZE[case["residual"]]
    side = 4 * h * (2 if case["post"] else 1) + (4 * t if case["gate"] else 0)
    moved = t * h * 2 * (s + e) + side
    if case["backward"]:
        moved += t * h * 3 * (s + e) + 2 * side
    return {"bytes": moved, "flops": (30.0 if case["backward"] else 10.0) * t * h}


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------

def _by_expert(state, a, product, cols):
    """product(rows of `a`, expert) for each expert's rows, in order."""
    out = torch.empty((state["rows"], cols), dtype=torch.float64, device="cuda")
    lo = 0
    for i, m in enumerate(state["splits"]):
        if m:
            out[lo:lo + m] = product(a[lo:lo + m].double(), i)
        lo += m
    return out


def _exact_gated(case, state):
    f = case["ffn"]
    rows = torch.index_select(state["x"], 0, state["row_index"])
    h = _by_expert(state, rows, lambda a, i: torch.matmul(a, state["w"][i].double().T), 2 * f)
    got = {"a": torch.nn.functional.silu(h[:, :f]) * h[:, f:]}
    if case["keep_h"]:
        got["h"] = h
    return got


def _exact_gated_bwd(case, state):
    f = case["ffn"]
    da = _by_expert(state, state["dy"], lambda a, i: torch.matmul(a, state["w"][i].double()), f)
    gate, up = state["h"][:, :f].double(), state["h"][:, f:].double()
    s = torch.sigmoid(gate)
    dh = torch.empty((state["rows"], 2 * f), dtype=torch.float64, device="cuda")
    # silu'(g) = s + g s (1 - s)
    dh[:, :f] = da * up * (s + gate * s * torch.sigmoid(-gate))
    dh[:, f:] = da * torch.nn.functional.silu(gate)
    return {"dh": dh, "a": torch.nn.functional.silu(gate) * up}


def _codes():
    """The finite e4m3 values from 0 up: 8 subnormal ones, then 8 to each power of two."""
    low = [m / 512 for m in range(8)]
    high = [(8 + m) * 2.0 ** (e - 9) for e in range(14) for m in range(8)] + \
        [(8 + m) * 32.0 for m in range(7)]
    return torch.tensor(low + high, dtype=torch.float64, device="cuda")


def _nearest(v):
    """Each value's code by search: the middle between two codes goes to the even one."""
    codes = _codes()
    at = torch.searchsorted((codes[1:] + codes[:-1]) / 2, v.abs())
    middle = torch.cat([(codes[1:] + codes[:-1]) / 2, codes[-1:] * 2])
    at += ((v.abs() == middle[at]) & (at % 2 == 1)).long()   # `at` is the code below a middle
    return torch.copysign(codes[at], v)


def _exact_fp8(case, state):
    t, k, n = case["tokens"], case["k"], case["n"]
    x = torch.zeros((t, k), dtype=torch.float64, device="cuda")
    for lo in range(0, k, 128):
        part = state["x"][:, lo:lo + 128].double()
        scale = (part.abs().max(dim=1, keepdim=True).values / 448).float().double()
        x[:, lo:lo + 128] = _nearest(part / torch.where(scale == 0, 1.0, scale)) * scale
    row, col = torch.arange(n, device="cuda") // 128, torch.arange(k, device="cuda") // 128

    def product(a, i):
        return torch.matmul(a, (state["wq"][i].double() * state["ws"][i].double()[row][:, col]).T)
    return _by_expert(state, x[state["row_index"].long()], product, n)


def _exact_fp8_weights(case, state):
    g, n, k = case["experts"], case["n"], case["k"]
    q = torch.empty((g, n, k), dtype=torch.float64, device="cuda")
    scale = torch.empty((g, -(-n // 128), -(-k // 128)), dtype=torch.float64, device="cuda")
    for i in range(g):
        for b, lo in enumerate(range(0, n, 128)):
            part = state["w"][i, lo:lo + 128].double()
            top = torch.stack([p.abs().max() for p in part.split(128, dim=1)])
            scale[i, b] = top / 448
            stored = (top / 448).float().double()
            over = torch.where(stored == 0, 1.0, stored).repeat_interleave(128)[:k]
            q[i, lo:lo + 128] = _nearest(part / over)
    return {"q": q, "scale": scale}


def _exact_norm(case, state):
    h = case["hidden"]
    f = state["f"].double()
    inv = 1.0 / torch.sqrt(torch.linalg.vecdot(f, f) / h + _EPS)
    b = f * inv[:, None] * state["post"].double() if case["post"] else f
    gate = state["gate"].double() if case["gate"] else torch.ones(len(f), device="cuda").double()
    exact_r = state["scale"] * state["x"].double() + gate[:, None] * b
    r = exact_r.to(state["x"].dtype).double()         # as it is stored
    inv_r = 1.0 / torch.sqrt(torch.linalg.vecdot(r, r) / h + _EPS)
    pre = state["pre"].double()
    got = {"r": exact_r, "y": r * inv_r[:, None] * pre}
    if case["backward"]:
        dy = state["dy"].double()
        u = dy * pre
        total = state["dr"].double() + inv_r[:, None] * u
        total -= (inv_r ** 3 * torch.linalg.vecdot(u, r) / h)[:, None] * r
        got["dx"] = state["scale"] * total
        got["dpre"] = torch.einsum("th,th,t->h", dy, r, inv_r)
        db = gate[:, None] * total
        got["df"] = db
        if case["post"]:
            got["dpost"] = torch.einsum("th,th,t->h", db, f, inv)
            u = db * state["post"].double()
            got["df"] = inv[:, None] * u - (inv ** 3 * torch.linalg.vecdot(u, f) / h)[:, None] * f
        if case["gate"]:
            got["dgate"] = torch.linalg.vecdot(total, b)
    return got


def exact(case, seed):
    state = prepare(case, seed)
    return {"gated": _exact_gated, "gated_bwd": _exact_gated_bwd, "fp8": _exact_fp8,
            "fp8_weights": _exact_fp8_weights, "norm": _exact_norm}[case["op"]](case, state)
