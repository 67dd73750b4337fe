"""The norms around a block with its gate and the residual scale, and their gradients,
against the formulas in float64."""

import math

import pytest
import torch

import moe_expert_grouped_group_amd as mx

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24    # a rounding to fp32


def _draw(shape, seed, dtype=F32, std=1.0):
    gen = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").mul_(std).to(dtype)


def _case(t, h, dtype, x_dtype, post, gate, pre, w_dtype=F32, seed=1):
    loud = torch.where(_draw((h,), seed + 8) > 2, 20.0, 1.0)
    return dict(x=(_draw((t, h), seed, std=2.0) * loud).to(x_dtype), f=_draw((t, h), seed + 1, dtype, 0.7),
                gate=torch.sigmoid(_draw((t,), seed + 2)) if gate else None,
                post_weight=(1 + 0.3 * _draw((h,), seed + 3)).to(w_dtype) if post else None,
                pre_weight=(1 + 0.3 * _draw((h,), seed + 4)).to(w_dtype) if pre else None)


def _near(got, ref, off, what):
    fin = torch.finfo(got.dtype)
    tol = off + (ref.abs() + off) * fin.eps / 2 + fin.tiny * fin.eps
    assert not torch.isnan(got).any(), what
    bad = (got.double() - ref).abs() > tol
    assert not bad.any(), (what, int(bad.sum()), float(((got.double() - ref).abs() / tol).max()))


# A row's sum of H terms: at most 16 terms a lane one after the other, then 10 steps over the
# lanes and waves, each a rounding; every term itself takes up to 3.
SUM = 30 * U


def _inverse(v, eps):
    """1 / sqrt(mean v^2 + eps) and its relative error: half of the sum's (all terms of one sign),
    the mean, eps and the hardware's 1 ulp (2 U)."""
    return 1 / torch.sqrt((v * v).mean(1, keepdim=True) + eps), SUM / 2 + 6 * U


def _check(case, scale, eps, r, y, dy=None, dr=None, grad=None):
    x, f, gate, post, pre = (None if case[n] is None else case[n].double()
                             for n in ("x", "f", "gate", "post_weight", "pre_weight"))
    h = x.shape[1]
    g = torch.ones((len(x), 1), dtype=torch.float64, device="cuda") if gate is None else gate[:, None]
    if f is not None:
        b, eb = f, 0.0
        if post is not None:
            inv, e = _inverse(f, eps)
            b, eb = f * inv * post, e + 4 * U
        ref = scale * x + g * b
        _near(r, ref, (scale * x).abs() * 2 * U + (g * b).abs() * (eb + 3 * U) + ref.abs() * 2 * U, "r")
    else:
        assert r is case["x"]
    stored = r.double()
    inv_r, e_r = _inverse(stored, eps)
    if pre is not None:
        want = stored * inv_r * pre
        _near(y, want, want.abs() * (e_r + 4 * U), "y")
    if grad is None:
        return
    total = torch.zeros_like(x) if dr is None else dr.double()
    size = total.abs()
    if dy is not None:
        u = dy.double() * pre
        mean = (u * stored).mean(1, keepdim=True)
        total = total + inv_r * u - inv_r ** 3 * mean * stored
        # the mean's terms may cancel: its error goes by their sizes
        e_mean = (u * stored).abs().mean(1, keepdim=True) * (SUM + 4 * U)
        e_total = (inv_r * u).abs() * (e_r + 4 * U) + stored.abs() * inv_r ** 3 * (
            e_mean + mean.abs() * (3 * e_r + 6 * U))
        size = size + (inv_r * u).abs() + (inv_r ** 3 * mean * stored).abs()
    else:
        e_total = torch.zeros_like(x)
    e_total = e_total + size * 3 * U
    k = scale if f is not None else 1.0
    _near(grad.x, k * total, abs(k) * e_total + (k * total).abs() * U, "dx")
    # column sums: rows one after the other in a workgroup, then the workgroups'
    steps = (len(x) / 16 + 40) * U
    if pre is not None and dy is not None:
        term = dy.double() * stored * inv_r
        _near(grad.pre_weight, term.sum(0), term.abs().sum(0) * (steps + e_r + 4 * U), "dpre")
    if f is None:
        return
    db, e_db = g * total, g.abs() * e_total + (g * total).abs() * U
    if gate is not None:
        bt = f * (inv * post if post is not None else 1.0)
        off = (total * bt).abs().sum(1) * (SUM + eb + 6 * U) + (e_total * bt.abs()).sum(1)
        _near(grad.gate, (total * bt).sum(1), off, "dgate")
    if post is None:
        _near(grad.f, db, e_db, "df")
        return
    inv, e_f = _inverse(f, eps)
    term = db * f * inv
    _near(grad.post_weight, term.sum(0),
          term.abs().sum(0) * (steps + e_f + 4 * U) + (e_db * (f * inv).abs()).sum(0), "dpost")
    u, e_u = db * post, e_db * post.abs() + (db * post).abs() * 2 * U
    mean = (u * f).mean(1, keepdim=True)
    e_mean = (u * f).abs().mean(1, keepdim=True) * (SUM + 4 * U) + (e_u * f.abs()).mean(1, keepdim=True)
    want = inv * u - inv ** 3 * mean * f
    off = inv * e_u + (inv * u).abs() * (e_f + 4 * U) + f.abs() * inv ** 3 * (e_mean + mean.abs() * (3 * e_f + 6 * U))
    _near(grad.f, want, off + ((inv * u).abs() + (inv ** 3 * mean * f).abs()) * 2 * U, "df")


SIZES = [(1, 1), (1, 7), (3, 8), (5, 64), (70, 129), (33, 512), (7, 513), (9, 1024), (300, 1031), (5, 2048), (3, 2056),
         (4, 4096), (6, 4100), (5, 7168), (3, 8192), (2, 8199), (3, 16384), (2, 16383)]


@pytest.mark.parametrize("dtype,x_dtype", [(BF, BF), (BF, F32), (HF, HF), (HF, F32)])
@pytest.mark.parametrize("t,h", SIZES)
def test_step(t, h, dtype, x_dtype):
    """Everything at once: both norms, gate, residual scale, all gradients."""
    case = _case(t, h, dtype, x_dtype, True, True, True)
    kw = {k: v for k, v in case.items() if k not in ("x", "f")}
    r, y = mx.residual_norm(case["x"], case["f"], residual_scale=0.75, **kw)
    assert r.dtype == x_dtype and y.dtype == dtype
    dy, dr = _draw((t, h), 20, dtype), _draw((t, h), 21, x_dtype)
    grad = mx.residual_norm_bwd(dy, dr, r, case["f"], residual_scale=0.75, **kw)
    _check(case, 0.75, 1e-6, r, y, dy, dr, grad)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("pre", [True, False])
@pytest.mark.parametrize("with_dr", [True, False])
@pytest.mark.parametrize("t,h", [(37, 200), (6, 2500)])
def test_parts(t, h, post, gate, pre, with_dr):
    """Each part left out."""
    case = _case(t, h, BF, BF, post, gate, pre, w_dtype=BF)
    kw = {k: v for k, v in case.items() if k not in ("x", "f")}
    r, y = mx.residual_norm(case["x"], case["f"], eps=1e-3, **kw)
    assert (y is None) == (not pre)
    if not pre and not with_dr:
        return
    dy, dr = _draw((t, h), 20, BF) if pre else None, _draw((t, h), 21, BF) if with_dr else None
    grad = mx.residual_norm_bwd(dy, dr, r, case["f"], eps=1e-3, **kw)
    assert (grad.gate is None) == (not gate) and (grad.post_weight is None) == (not post)
    assert (grad.pre_weight is None) == (not pre)
    _check(case, 1.0, 1e-3, r, y, dy, dr, grad)


@pytest.mark.parametrize("dtype,x_dtype", [(BF, BF), (HF, F32)])
@pytest.mark.parametrize("t,h", [(1, 1), (40, 333), (3, 5000)])
def test_before_the_first_block(t, h, dtype, x_dtype):
    """Without f: the norm of x alone."""
    case = _case(t, h, dtype, x_dtype, False, False, True)
    case["f"] = None
    r, y = mx.residual_norm(case["x"], pre_weight=case["pre_weight"], out_dtype=dtype)
    dy = _draw((t, h), 20, dtype)
    for dr in (None, _draw((t, h), 21, x_dtype)):
        grad = mx.residual_norm_bwd(dy, dr, r, pre_weight=case["pre_weight"])
        assert grad.f is None and grad.gate is None
        _check(case, 1.0, 1e-6, r, y, dy, dr, grad)


@pytest.mark.parametrize("x_dtype", [BF, F32])
@pytest.mark.parametrize("power", [55, -60])
@pytest.mark.parametrize("t,h", [(5, 96), (300, 1031), (4, 4096)])
def test_loud_and_quiet_rows(t, h, power, x_dtype):
    """Rows whose squares are fp32 numbers and whose inverse norms' cubes are not."""
    s = 2.0 ** power
    case = _case(t, h, BF, x_dtype, True, True, True)
    case["x"], case["f"] = case["x"] * s, case["f"] * s
    case["gate"] = case["gate"] * s
    kw = {k: v for k, v in case.items() if k not in ("x", "f")}
    r, y = mx.residual_norm(case["x"], case["f"], residual_scale=0.5, eps=0.0, **kw)
    dy, dr = _draw((t, h), 20, BF), _draw((t, h), 21, x_dtype) / s
    grad = mx.residual_norm_bwd(dy, dr, r, case["f"], residual_scale=0.5, eps=0.0, **kw)
    _check(case, 0.5, 0.0, r, y, dy, dr, grad)


@pytest.mark.parametrize("t,h", [(5000, 64), (3000, 1000), (700, 2048), (600, 4096), (300, 8192)])
def test_many_rows(t, h):
    """More rows than one to each workgroup: column sums over several."""
    case = _case(t, h, BF, BF, True, True, True)
    kw = {k: v for k, v in case.items() if k not in ("x", "f")}
    r, y = mx.residual_norm(case["x"], case["f"], residual_scale=-1.5, **kw)
    dy, dr = _draw((t, h), 20, BF), _draw((t, h), 21, BF)
    grad = mx.residual_norm_bwd(dy, dr, r, case["f"], residual_scale=-1.5, **kw)
    _check(case, -1.5, 1e-6, r, y, dy, dr, grad)
    again = mx.residual_norm_bwd(dy, dr, r, case["f"], residual_scale=-1.5, **kw)
    for name in ("x", "f", "gate", "post_weight", "pre_weight"):
        assert torch.equal(getattr(grad, name), getattr(again, name)), name


def test_rows_of_zeros_and_no_numbers():
    """A row of zeros with eps gives zeros; infinities and NaN stay in their row, gate 0 or not."""
    t, h = 5, 300
    case = _case(t, h, BF, BF, True, True, True)
    kw = {k: v for k, v in case.items() if k not in ("x", "f")}
    case["x"][0], case["f"][0] = 0, 0
    case["f"][2, 7], case["x"][3, 1] = math.nan, math.inf
    r, y = mx.residual_norm(case["x"], case["f"], **kw)
    assert (r[0] == 0).all() and (y[0] == 0).all()
    assert torch.isnan(r[2]).all() and torch.isinf(r[3, 1])
    assert torch.isfinite(r[[0, 1, 4]].float()).all() and torch.isfinite(y[[0, 1, 4]].float()).all()
    dy, dr = _draw((t, h), 20, BF), _draw((t, h), 21, BF)
    grad = mx.residual_norm_bwd(dy, dr, r, case["f"], **kw)
    assert torch.isfinite(grad.x[[0, 1, 4]].float()).all() and torch.isnan(grad.x[2]).any()


@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("h", [8, 300, 1031, 4096, 9000])
@pytest.mark.parametrize("dtype,x_dtype", [(BF, BF), (BF, F32), (HF, HF)])
def test_no_numbers_in_an_output_without_its_norm(dtype, x_dtype, h, gate):
    """f without a norm of its own reaches no gradient but the gate's: df = gate dr, whatever f holds."""
    t = 7
    case = _case(t, h, dtype, x_dtype, False, gate, False)
    f, gates = case["f"], case["gate"]
    f[1, h - 1], f[2], f[3, 0] = math.inf, math.nan, -math.inf
    dr = _draw((t, h), 21, x_dtype)
    r, _ = mx.residual_norm(case["x"], f, residual_scale=0.5, gate=gates)
    grad = mx.residual_norm_bwd(None, dr, r, f, residual_scale=0.5, gate=gates)
    g = 1.0 if gates is None else gates[:, None]
    assert torch.equal(grad.f, (g * dr.float()).to(dtype))
    assert torch.equal(grad.x, (0.5 * dr.float()).to(x_dtype))
    if gate:
        assert torch.isfinite(grad.gate[[0, 4, 5, 6]]).all() and not torch.isfinite(grad.gate[1:4]).any()


def test_in_place_and_buffers():
    """r may be x; dx may be dr, df may be dy or f."""
    t, h = 40, 520
    case = _case(t, h, BF, BF, True, True, True)
    kw = {k: v for k, v in case.items() if k not in ("x", "f")}
    r, y = mx.residual_norm(case["x"], case["f"], **kw)
    x = case["x"].clone()
    got = mx.residual_norm(x, case["f"], r=x, y=torch.empty_like(y), **kw)
    assert got[0] is x and torch.equal(x, r) and torch.equal(got[1], y)
    dy, dr = _draw((t, h), 20, BF), _draw((t, h), 21, BF)
    want = mx.residual_norm_bwd(dy, dr, r, case["f"], **kw)
    ws = torch.empty(mx.residual_norm_bwd_workspace_bytes(t, h), dtype=torch.uint8, device="cuda")
    for which in ("dy", "f"):
        a, b, f = dr.clone(), dy.clone(), case["f"].clone()
        out = mx.ResidualNormGrad(x=a, f=b if which == "dy" else f)
        grad = mx.residual_norm_bwd(b, a, r, f, out=out, workspace=ws, **kw)
        assert grad.x is a
        for name in ("x", "f", "gate", "post_weight", "pre_weight"):
            assert torch.equal(getattr(grad, name), getattr(want, name)), (which, name)


@pytest.mark.parametrize("shift", [1, 3])
@pytest.mark.parametrize("h", [64, 1000, 4104])
def test_shifted_buffers(h, shift):
    """Rows that start off 16 bytes; what lies around the outputs stays."""
    t = 9
    case = _case(t, h, BF, BF, True, True, True)
    kw = {k: v for k, v in case.items() if k not in ("x", "f")}
    r, y = mx.residual_norm(case["x"], case["f"], **kw)

    def moved(src):
        buf = torch.full((t * h + 2 * shift,), 7.0, dtype=src.dtype, device="cuda")
        view = buf[shift:shift + t * h].view(t, h)
        view.copy_(src)
        return buf, view

    x, f = moved(case["x"])[1], moved(case["f"])[1]
    rb, rv = moved(torch.zeros_like(r))
    yb, yv = moved(torch.zeros_like(y))
    mx.residual_norm(x, f, r=rv, y=yv, **kw)
    assert torch.equal(rv, r) and torch.equal(yv, y)
    dy, dr = _draw((t, h), 20, BF), _draw((t, h), 21, BF)
    want = mx.residual_norm_bwd(dy, dr, r, case["f"], **kw)
    xb, xv = moved(torch.zeros_like(r))
    fb, fv = moved(torch.zeros_like(r))
    grad = mx.residual_norm_bwd(moved(dy)[1], moved(dr)[1], rv, f, out=mx.ResidualNormGrad(x=xv, f=fv), **kw)
    assert torch.equal(xv, want.x) and torch.equal(fv, want.f) and torch.equal(grad.pre_weight, want.pre_weight)
    for buf in (rb, yb, xb, fb):
        assert (buf[:shift] == 7.0).all() and (buf[-shift:] == 7.0).all()


def test_gradients_against_differences():
    """Central differences of <y, dy> + <r, dr> in float64 along random directions; the residual
    stream in fp32, so that its rounding does not count."""
    t, h = 11, 96
    case = _case(t, h, HF, F32, True, True, True)
    kw = {k: v for k, v in case.items() if k not in ("x", "f")}
    dy, dr = _draw((t, h), 20, HF), _draw((t, h), 21, F32)
    r, _ = mx.residual_norm(case["x"], case["f"], residual_scale=0.9, **kw)
    grad = mx.residual_norm_bwd(dy, dr, r, case["f"], residual_scale=0.9, **kw)

    def loss(x, f, gate, post_weight, pre_weight):
        n = lambda v: v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6)  # noqa: E731
        r = 0.9 * x + gate[:, None] * n(f) * post_weight
        return (n(r) * pre_weight * dy.double()).sum() + (r * dr.double()).sum()

    at = {k: v.double() for k, v in case.items()}
    for name in at:
        for seed in range(3):
            step = _draw(at[name].shape, 100 + seed).double()
            lo, hi = dict(at), dict(at)
            lo[name], hi[name] = at[name] - 1e-5 * step, at[name] + 1e-5 * step
            slope = float(loss(**hi) - loss(**lo)) / 2e-5
            got = getattr(grad, name).double()
            # df is rounded to fp16 (2^-11 of each value); the rest is fp32, r rounded to fp32 before
            # its norm: 200 roundings are more than lie on any path
            share = 2.0 ** -11 if name == "f" else 0.0
            off = float((got.abs() * step.abs()).sum()) * (share + 200 * U) + 1e-6 * abs(slope)
            assert abs(float((got * step).sum()) - slope) <= off, name


def test_no_rows():
    x = torch.zeros((0, 64), dtype=BF, device="cuda")
    w = torch.ones(64, device="cuda")
    g = torch.zeros(0, device="cuda")
    r, y = mx.residual_norm(x, x, gate=g, post_weight=w, pre_weight=w)
    assert r.shape == y.shape == (0, 64)
    grad = mx.residual_norm_bwd(x, x, r, x, gate=g, post_weight=w, pre_weight=w)
    assert grad.x.shape == (0, 64) and (grad.pre_weight == 0).all() and (grad.post_weight == 0).all()


def test_captured_and_replayed():
    t, h = 500, 1536
    case = _case(t, h, BF, BF, True, True, True)
    kw = {k: v for k, v in case.items() if k not in ("x", "f")}
    dy, dr = _draw((t, h), 20, BF), _draw((t, h), 21, BF)
    new = lambda *s, d=BF: torch.empty(s, dtype=d, device="cuda")  # noqa: E731
    r, y = new(t, h), new(t, h)
    out = mx.ResidualNormGrad(new(t, h), new(t, h), new(t, d=F32), new(h, d=F32), new(h, d=F32))
    ws = torch.empty(mx.residual_norm_bwd_workspace_bytes(t, h), dtype=torch.uint8, device="cuda")

    def step():
        mx.residual_norm(case["x"], case["f"], r=r, y=y, **kw)
        mx.residual_norm_bwd(dy, dr, r, case["f"], out=out, workspace=ws, **kw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    names = ("x", "f", "gate", "post_weight", "pre_weight")
    for seed in range(3):
        case["x"].copy_(_draw((t, h), 30 + seed, BF))
        dy.copy_(_draw((t, h), 40 + seed, BF))
        graph.replay()
        got = [t.clone() for t in (r, y, *(getattr(out, n) for n in names))]
        r2, y2 = mx.residual_norm(case["x"], case["f"], **kw)
        want = mx.residual_norm_bwd(dy, dr, r2, case["f"], **kw)
        torch.cuda.synchronize()
        for a, b in zip(got, (r2, y2, *(getattr(want, n) for n in names))):
            assert torch.equal(a, b)


@pytest.mark.parametrize("t,h", [(1, 16), (37, 127), (1000, 128), (50, 130), (333, 256), (9, 257)])
def test_short_rows(t, h):
    """Rows of 16 and 32 lanes, several to a wave; the last wave's rows not all there."""
    case = _case(t, h, HF, F32, True, True, True)
    kw = {k: v for k, v in case.items() if k not in ("x", "f")}
    r, y = mx.residual_norm(case["x"], case["f"], residual_scale=0.75, **kw)
    _check(case, 0.75, 1e-6, r, y)
