"""What is timed of the operators for experts with ragged token counts.

Three operators of a mixture-of-experts layer whose experts get any number of
token rows (the MXFP8 products of this package take runs of 128):

  product  the products grouped by expert of bf16 / fp16 tensors: forward (NT),
           gradient of the input (NN), gradient of the weight (TN)
  int8     tokens quantized to 8-bit integers with a scale each, and their
           product with weights that have a scale for each output channel
  routing  the k best experts of each token with their weights, the order of
           the rows by expert, the weighted sum of the experts' rows, and the
           gradients of both

`own` chooses between the plain torch form of each and the package's calls.
"""

import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "fp16": 2, "f32": 4}

# What a drawn case may cost at most: the largest listed product, and weights
# that leave room for several sets of inputs.
_FLOPS = 2 * 16384 * 4096 * 14336
_WEIGHTS = 1 << 29


def _product(name, layout, dtype, out, experts, active, tokens, top_k, k, n):
    """One product: tokens * top_k rows; `active` experts have rows, the others none.
    gather: row r of the product is token row_index[r] (otherwise the rows lie in order)."""
    return {"name": name, "op": "product", "layout": layout, "dtype": dtype, "out": out,
            "experts": experts, "active": active, "tokens": tokens, "top_k": top_k,
            "k": k, "n": n, "gather": layout != "NN"}


def _int8(name, dtype, out, experts, active, tokens, top_k, k, n):
    return {"name": name, "op": "int8", "dtype": dtype, "out": out, "experts": experts,
            "active": active, "tokens": tokens, "top_k": top_k, "k": k, "n": n}


def _route(name, dtype, tokens, experts, top_k, renormalize, masked, backward):
    return {"name": name, "op": "route", "dtype": dtype, "tokens": tokens, "experts": experts,
            "top_k": top_k, "renormalize": renormalize, "masked": masked, "backward": backward}


def _join(name, dtype, tokens, top_k, hidden, backward):
    return {"name": name, "op": "join", "dtype": dtype, "tokens": tokens, "top_k": top_k,
            "hidden": hidden, "backward": backward}


def listed():
    return [
        # training of an 8-expert layer (hidden 4096, FFN 14336): 8192 tokens,
        # two experts each, as many rows as the gate happens to send
        _product("forward 8x4096x14336", "NT", "bf16", "bf16", 8, 8, 8192, 2, 4096, 14336),
        _product("input grad 8x4096x14336", "NN", "bf16", "bf16", 8, 8, 8192, 2, 4096, 14336),
        # the weight gradient of the same layer, kept in fp32
        _product("weight grad 8x4096x14336", "TN", "bf16", "f32", 8, 8, 8192, 2, 4096, 14336),
        # many experts under skewed routing, 38 of 128 with no token
        _product("forward 128x7168x2048", "NT", "fp16", "fp16", 128, 90, 4096, 8, 7168, 2048),
        # nothing is a multiple of anything: a small odd model
        _product("forward odd 5x1031x517", "NT", "fp16", "f32", 5, 4, 1777, 1, 1031, 517),
        # decoding 8 sequences: a row or two for each expert
        _product("decode 8x4096x14336", "NT", "bf16", "bf16", 8, 7, 8, 2, 4096, 14336),
        # serving in 8-bit integers: a prompt batch
        _int8("int8 prompt 8x4096x14336", "bf16", "bf16", 8, 8, 8192, 2, 4096, 14336),
        # 8 sequences decoded over many experts, eight for each token
        _int8("int8 decode 128x7168x2048", "bf16", "bf16", 128, 48, 8, 8, 7168, 2048),
        # one token through one dense linear of odd width: latency
        _int8("int8 dense 1x1000x4099", "fp16", "f32", 1, 1, 1, 1, 1000, 4099),
        # the gate of a training step: choice, order of the rows, gradient
        _route("route 32768x128 step", "f32", 32768, 128, 8, True, True, True),
        # the gate for a handful of decoded tokens: latency
        _route("route 5x256", "bf16", 5, 256, 8, False, False, False),
        # the experts' rows summed for each token, and the gradients of that
        _join("join 16384x8x4096 step", "bf16", 16384, 8, 4096, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A feature count: mostly a multiple of 8, one in four any number."""
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.25 else max(8, v // 8 * 8)


def _sizes(rng):
    """Rows and weights of a drawn product within what the largest listed one costs."""
    k, n = _width(rng, 128, 8192), _width(rng, 128, 14336)
    experts = _log(rng, 1, max(1, min(256, _WEIGHTS // (k * n))))
    top_k = min(experts, rng.choice([1, 1, 2, 4, 8]))
    most = max(1, int(_FLOPS / (2.0 * k * n * top_k)))
    tokens = _log(rng, 1, max(1, min(32768 // top_k, most)))
    active = rng.randint(max(1, min(experts, tokens * top_k) // 2), min(experts, tokens * top_k))
    return experts, active, tokens, top_k, k, n


def draw(rng):
    kind = rng.choice(["product", "product", "int8", "route", "join"])
    if kind == "product":
        dtype = rng.choice(["bf16", "fp16"])
        case = _product("", rng.choice(["NT", "NN", "TN"]), dtype, rng.choice([dtype, "f32"]),
                        *_sizes(rng))
    elif kind == "int8":
        case = _int8("", rng.choice(["bf16", "fp16"]), rng.choice(["bf16", "fp16", "f32"]),
                     *_sizes(rng))
    elif kind == "route":
        experts = _log(rng, 2, 512)
        case = _route("", rng.choice(["f32", "bf16", "fp16"]), _log(rng, 1, 131072), experts,
                      rng.randint(1, min(8, experts)), rng.random() < 0.5, rng.random() < 0.5,
                      rng.random() < 0.5)
    else:
        top_k = rng.choice([1, 2, 4, 6, 8])
        case = _join("", rng.choice(["bf16", "fp16"]), _log(rng, 1, 131072 // top_k), top_k,
                     _width(rng, 64, 8192), rng.random() < 0.5)
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


def prepare(case, seed):
    dtype = _TYPES[case["dtype"]]
    state = {"case": case}
    if case["op"] == "product":
        state |= _rows(case, seed)
        g, k, n = case["experts"], case["k"], case["n"]
        if case["layout"] != "NN":
            state["x"] = _normal((case["tokens"], k), seed + 1, dtype)
        if case["layout"] != "TN":
            state["w"] = _normal((g, n, k), seed + 2, dtype, 0.02)
        if case["layout"] != "NT":
            state["dy"] = _normal((state["rows"], n), seed + 3, dtype)
    elif case["op"] == "int8":
        state |= _rows(case, seed)
        g, k, n = case["experts"], case["k"], case["n"]
        state["x"] = _normal((case["tokens"], k), seed + 1, dtype)
        gen = torch.Generator("cuda").manual_seed(seed + 2)
        state["wq"] = torch.randint(-127, 128, (g, n, k), generator=gen, device="cuda",
                                    dtype=torch.int8)
        state["ws"] = torch.rand((g, n), generator=gen, device="cuda") * 4e-4 + 1e-4
    elif case["op"] == "route":
        t, e = case["tokens"], case["experts"]
        gen = torch.Generator("cuda").manual_seed(seed)
        logits = torch.randn((t, e), generator=gen, device="cuda") * 1.5
        logits += torch.randn((1, e), generator=gen, device="cuda")   # experts differ in favour
        state["mask"] = None
        if case["masked"]:
            # padding tokens hold anything; experts out of service are at -inf
            mask = torch.rand(t, generator=gen, device="cuda") < 0.9
            logits[~mask] = math.nan
            out = torch.rand(e, generator=gen, device="cuda") < 0.05
            out[torch.argsort(out.int(), stable=True)[:case["top_k"]]] = False
            logits[:, out] = -math.inf
            state["mask"] = mask
        state["logits"] = logits.to(dtype)
        state["dweights"] = torch.randn((t, case["top_k"]), generator=gen, device="cuda")
    else:
        t, top_k, h = case["tokens"], case["top_k"], case["hidden"]
        gen = torch.Generator("cuda").manual_seed(seed)
        state["y"] = _normal((t * top_k, h), seed + 1, dtype)
        state["pos"] = torch.randperm(t * top_k, generator=gen, device="cuda").view(t, top_k).int()
        state["weights"] = torch.rand((t, top_k), generator=gen, device="cuda")
        state["dout"] = _normal((t, h), seed + 2, dtype)
    return state


# ----------------------------------------------------------------------------
# the plain forms
# ----------------------------------------------------------------------------

def _plain_product(state):
    case, splits = state["case"], state["splits"]
    out = _TYPES[case["out"]]
    index = state["row_index"].long()
    if case["layout"] == "NT":
        parts = zip(state["x"][index].split(splits), state["w"])
        return torch.cat([x.float() @ w.float().t() for x, w in parts]).to(out)
    if case["layout"] == "NN":
        parts = zip(state["dy"].split(splits), state["w"])
        return torch.cat([dy.float() @ w.float() for dy, w in parts]).to(out)
    parts = zip(state["dy"].split(splits), state["x"][index].split(splits))
    return torch.stack([dy.float().t() @ x.float() for dy, x in parts]).to(out)


def _plain_int8(state):
    case = state["case"]
    # the stored scale is the fp32 value nearest to amax / 127, and a quotient next to
    # the border between two integers is decided in 64 bits
    scale = (state["x"].abs().amax(1).double() / 127).float()
    q = (state["x"].double() / scale.double()[:, None]).round().float()
    index = state["row_index"].long()
    parts = zip(q[index].split(state["splits"]), state["wq"], state["ws"])
    y = torch.cat([(a @ w.float().t()) * s for a, w, s in parts])
    return (y * scale[index][:, None]).to(_TYPES[case["out"]])


def _plain_route(state):
    case = state["case"]
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    logits = state["logits"].float()
    if state["mask"] is not None:
        logits = logits.masked_fill(~state["mask"][:, None], -math.inf)
    value, order = torch.sort(logits, dim=1, descending=True, stable=True)
    live = value[:, :k] > -math.inf
    ids = torch.where(live, order[:, :k], -1)
    top = torch.where(live[:, :1], value[:, :1], 0.0)
    p = torch.exp(value - top)
    total = p[:, :k].sum(1, keepdim=True) if case["renormalize"] else p.sum(1, keepdim=True)
    weights = torch.where(live, p[:, :k] / total, 0.0)
    # rows by expert, and by token within an expert
    flat = torch.where(live, ids, e).flatten()
    rows = torch.argsort(flat, stable=True)
    m_splits = torch.bincount(flat, minlength=e + 1)[:e]
    routed = flat[rows] < e
    row_token = torch.where(routed, rows // k, -1).int()
    pos = torch.empty_like(rows)
    pos[rows] = torch.where(routed, torch.arange(t * k, device=rows.device), -1)
    got = {"ids": ids.int(), "weights": weights, "m_splits": m_splits, "row_token": row_token,
           "row_pos": pos.view(t, k).int()}
    if case["backward"]:
        dw = torch.where(live, state["dweights"], 0.0)
        inner = (dw * weights).sum(1, keepdim=True)
        if case["renormalize"]:
            grad = torch.zeros_like(logits)
        else:
            grad = -inner * torch.exp(logits - top) / total
            grad = torch.where(live[:, :1], grad, 0.0)
        add = weights * (dw - inner) if case["renormalize"] else weights * dw
        grad.scatter_add_(1, torch.where(live, ids, 0), torch.where(live, add, 0.0))
        got["dlogits"] = grad.to(state["logits"].dtype)
    return got


def _plain_join(state):
    pos, w = state["pos"].long(), state["weights"]
    rows = state["y"].float()[pos]
    got = {"out": (rows * w[:, :, None]).sum(1).to(state["y"].dtype)}
    if state["case"]["backward"]:
        dout = state["dout"].float()
        dy = torch.empty_like(state["y"])
        dy[pos] = (dout[:, None, :] * w[:, :, None]).to(dy.dtype)
        got["dy"] = dy
        got["dweights"] = (rows * dout[:, None, :]).sum(2)
    return got


# ----------------------------------------------------------------------------
# the package's calls
# ----------------------------------------------------------------------------

def _own(state):
    import moe_expert_grouped_group_amd as mx
    case = state["case"]
    if case["op"] == "product":
        out = _TYPES[case["out"]]
        if case["layout"] == "NT":
            return mx.ragged_gemm("NT", state["x"], state["w"], state["m_splits"],
                                  row_index=state["row_index"], out_dtype=out)
        if case["layout"] == "NN":
            return mx.ragged_gemm("NN", state["dy"], state["w"], state["m_splits"], out_dtype=out)
        return mx.ragged_gemm("TN", state["dy"], state["x"], state["m_splits"],
                              row_index=state["row_index"], out_dtype=out)
    if case["op"] == "int8":
        q, scale = mx.quantize_int8(state["x"])
        return mx.ragged_gemm_int8(q, scale, state["wq"], state["ws"], state["m_splits"],
                                   row_index=state["row_index"], out_dtype=_TYPES[case["out"]])
    if case["op"] == "route":
        r = mx.moe_route(state["logits"], case["top_k"], renormalize=case["renormalize"],
                         token_mask=state["mask"])
        got = {"ids": r.ids, "weights": r.weights, "m_splits": r.m_splits,
               "row_token": r.row_token, "row_pos": r.row_pos}
        if case["backward"]:
            got["dlogits"] = mx.moe_route_bwd(state["logits"], r, state["dweights"])
        return got
    got = {"out": mx.moe_combine(state["y"], state["pos"], state["weights"])}
    if case["backward"]:
        got["dy"], got["dweights"] = mx.moe_combine_bwd(state["dout"], state["y"], state["pos"],
                                                        state["weights"])
    return got


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "product":
        return _plain_product(state)
    if op == "int8":
        return _plain_int8(state)
    return _plain_route(state) if op == "route" else _plain_join(state)


def work(case):
    """Each input read once, each output written once; the weights of experts
    without rows are not read."""
    if case["op"] in ("product", "int8"):
        t, r, k, n = case["tokens"], case["tokens"] * case["top_k"], case["k"], case["n"]
        g, active = case["experts"], case["active"]
        e, o = _SIZE[case["dtype"]], _SIZE[case["out"]]
        index = 0 if case.get("layout") == "NN" else 4 * r
        side = 8 * g + index
        if case["op"] == "int8":
            moved = t * k * e + active * n * (k + 4) + r * n * o
        elif case["layout"] == "NT":
            moved = t * k * e + active * n * k * e + r * n * o
        elif case["layout"] == "NN":
            moved = r * n * e + active * n * k * e + r * k * o
        else:
            moved = t * k * e + r * n * e + g * n * k * o
        return {"bytes": moved + side, "flops": 2.0 * r * k * n}
    if case["op"] == "route":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        moved = t * e * _SIZE[case["dtype"]] + 8 * e + 16 * t * k + (t if case["masked"] else 0)
        if case["backward"]:
            moved += t * e * _SIZE[case["dtype"]] + 4 * t * k
        return {"bytes": moved, "flops": 4.0 * t * e}
    t, k, h, e = case["tokens"], case["top_k"], case["hidden"], _SIZE[case["dtype"]]
    moved = (t * k + t) * h * e + 8 * t * k
    if case["backward"]:
        moved += (t + t * k) * h * e + 4 * t * k
    return {"bytes": moved, "flops": (6.0 if case["backward"] else 2.0) * t * k * h}


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------

def _exact_product(case, state):
    g, k, n = case["experts"], case["k"], case["n"]
    rows, token = state["rows"], state["row_index"].long()
    if case["layout"] == "TN":
        out = torch.zeros((g, n, k), dtype=torch.float64, device="cuda")
    else:
        out = torch.empty((rows, n if case["layout"] == "NT" else k), dtype=torch.float64,
                          device="cuda")
    lo = 0
    for i, m in enumerate(state["splits"]):
        at = slice(lo, lo + m)
        lo += m
        if m == 0:
            continue
        if case["layout"] == "NT":
            torch.matmul(state["x"][token[at]].double(), state["w"][i].double().T, out=out[at])
        elif case["layout"] == "NN":
            torch.matmul(state["dy"][at].double(), state["w"][i].double(), out=out[at])
        else:
            torch.matmul(state["dy"][at].double().T, state["x"][token[at]].double(), out=out[i])
    return out


def _exact_int8(case, state):
    # the scale is what is stored: amax / 127 in 32 bits; each code is the integer
    # nearest to the value over it, ties to the even one
    x = state["x"].double()
    scale = (x.abs().max(dim=1).values / 127).float().double()
    codes = torch.round(x / scale.unsqueeze(1))
    out = torch.empty((state["rows"], case["n"]), dtype=torch.float64, device="cuda")
    lo = 0
    for i, m in enumerate(state["splits"]):
        token = state["row_index"][lo:lo + m].long()
        if m:
            acc = torch.matmul(codes[token], state["wq"][i].double().T)
            out[lo:lo + m] = acc * scale[token].unsqueeze(1) * state["ws"][i].double()
        lo += m
    return out


def _exact_route(case, state):
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    z = state["logits"].double()
    if state["mask"] is not None:
        z[~state["mask"]] = -math.inf
    left, ids, chosen = z.clone(), [], torch.zeros_like(z, dtype=torch.bool)
    number = torch.arange(e, device=z.device)
    for _ in range(k):
        best = left.amax(1, keepdim=True)
        first = torch.where(left == best, number, e).amin(1)     # ties: the lowest index
        has = best[:, 0] > -math.inf
        ids.append(torch.where(has, first, -1))
        hit = (number == first[:, None]) & has[:, None]
        chosen |= hit
        left[hit] = -math.inf
    ids = torch.stack(ids, 1)
    live = ids >= 0
    over = torch.where(chosen, z, -math.inf) if case["renormalize"] else z
    some = live[:, 0]
    prob = torch.zeros_like(z)
    prob[some] = torch.softmax(over[some], 1)
    weights = torch.where(live, prob.gather(1, ids.clamp(min=0)), 0.0)
    # position of a choice: rows of lower experts, then earlier tokens of its own
    counts = chosen.sum(0)
    before = torch.cumsum(counts, 0) - counts
    place = before + torch.cumsum(chosen, 0) - 1
    pos = torch.where(live, place.gather(1, ids.clamp(min=0)), -1)
    row_token = torch.full((t * k,), -1, dtype=torch.int32, device=z.device)
    which = torch.arange(t, device=z.device)[:, None].expand(t, k)
    row_token[pos[live]] = which[live].int()
    got = {"ids": ids.int(), "weights": weights, "m_splits": counts, "row_token": row_token,
           "row_pos": pos.int()}
    if case["backward"]:
        # Jacobian of the softmax: p (d - <p, d>), with d the gradient at the chosen ones
        d = torch.zeros_like(z)
        d.scatter_add_(1, ids.clamp(min=0), torch.where(live, state["dweights"].double(), 0.0))
        got["dlogits"] = prob * (d - (prob * d).sum(1, keepdim=True))
    return got


def _exact_join(case, state):
    t, k, h = case["tokens"], case["top_k"], case["hidden"]
    w, dout = state["weights"].double(), state["dout"].double()
    out = torch.zeros((t, h), dtype=torch.float64, device="cuda")
    dw = torch.empty((t, k), dtype=torch.float64, device="cuda")
    dy = torch.zeros((t * k, h), dtype=torch.float64, device="cuda") if case["backward"] else None
    for j in range(k):
        at = state["pos"][:, j].long()
        y = state["y"][at].double()
        out += w[:, j, None] * y
        if case["backward"]:
            dw[:, j] = torch.linalg.vecdot(y, dout)
            dy[at] = w[:, j, None] * dout
    return {"out": out, "dy": dy, "dweights": dw} if case["backward"] else {"out": out}


def exact(case, seed):
    state = prepare(case, seed)
    return {"product": _exact_product, "int8": _exact_int8, "route": _exact_route,
            "join": _exact_join}[case["op"]](case, state)
