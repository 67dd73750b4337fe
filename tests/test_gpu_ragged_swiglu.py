"""The gated feed-forward block of ragged experts (both projections, activation and
product in one kernel; the backward pass inside the down projection's gradient)
against plain per-expert products in float64."""

import math

import pytest
import torch

import moe_expert_grouped_group_amd as mx

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def _normal(shape, seed, dtype, std=1.0):
    gen = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").mul_(std).to(dtype)


def _ms(splits):
    return torch.tensor(splits, dtype=torch.int64, device="cuda")


def _spans(splits, rows):
    lo, got = 0, []
    for m in splits:
        got.append((min(lo, rows), min(lo + max(m, 0), rows)))
        lo += max(m, 0)
    return got


def _gather(x, index):
    if index is None:
        return x.double()
    at = index.long()
    ok = (at >= 0) & (at < x.shape[0])
    if x.shape[0] == 0:
        return torch.zeros((at.numel(), x.shape[1]), dtype=torch.float64, device=x.device)
    return torch.where(ok[:, None], x[at.clamp(0, x.shape[0] - 1)].double(), 0.0)


def _sum_error(mag, terms):
    """A sum of `terms` exact products in fp32, in steps of at most 16 terms, each addition
    off by at most one fp32 step of the magnitude summed so far."""
    return mag * (terms / 16 + 20) * 2.0 ** -23


def _near(got, ref, off, what):
    """`off`: the error ahead of the rounding to got's type, which adds half a step (or half
    of the smallest subnormal step)."""
    fin = torch.finfo(got.dtype)
    tol = off + (ref.abs() + off) * fin.eps / 2 + fin.tiny * fin.eps
    assert not torch.isnan(got).any(), what
    bad = (got.double() - ref).abs() > tol
    assert not bad.any(), (what, int(bad.sum()), float(((got.double() - ref).abs() / tol).max()))


def _act_error(g):
    """Relative error of sigmoid(g) and of what is made of it: the exponent's rounding is
    |g| 2^-24 of it, the hardware's exponential and reciprocal 1 ulp (2^-23) each, and at
    most four roundings of 2^-24 follow.  The reciprocal gives 0 where its result is below
    the smallest normal fp32 number, 2^-126: the error is up to 1 of a sigmoid less than that
    (g < -87.3), which is an absolute 2^-126 of the sigmoid."""
    return (g.abs() * 1.5 + 8) * 2.0 ** -23 + torch.where(g < -87.3, 1.0, 0.0)


def _check_forward(x, w, splits, index, h, a, rows):
    f = w.shape[1] // 2
    for e, (lo, hi) in enumerate(_spans(splits, rows)):
        xr, we = _gather(x, index)[lo:hi], w[e].double()
        z = xr @ we.T
        ez = _sum_error(xr.abs() @ we.abs().T, x.shape[1])
        if h is not None:
            _near(h[lo:hi], z, ez, f"h of expert {e}")
        g, u, eg, eu = z[:, :f], z[:, f:], ez[:, :f], ez[:, f:]
        silu = g * torch.sigmoid(g)
        # |silu'| <= 1.1
        off = 1.1 * eg * (u.abs() + eu) + silu.abs() * eu + (silu * u).abs() * _act_error(g)
        _near(a[lo:hi], silu * u, off, f"a of expert {e}")


def _check_backward(dy, w, h, splits, dh, a):
    f = w.shape[2]
    for e, (lo, hi) in enumerate(_spans(splits, dy.shape[0])):
        d, we = dy[lo:hi].double(), w[e].double()
        da = d @ we
        ed = _sum_error(d.abs() @ we.abs(), dy.shape[1])
        g, u = h[lo:hi, :f].double(), h[lo:hi, f:].double()
        s = torch.sigmoid(g)
        silu, slope = g * s, s * (1 + g * (1 - s))
        # the slope's two terms may cancel: its error goes by their sizes
        eslope = s * (1 + g.abs()) * _act_error(g)
        _near(dh[lo:hi, :f], da * u * slope,
              u.abs() * (ed * (slope.abs() + eslope) + da.abs() * (eslope + slope.abs() * 2.0 ** -22)), f"dgate {e}")
        _near(dh[lo:hi, f:], da * silu, silu.abs() * (ed + da.abs() * _act_error(g)), f"dup {e}")
        if a is not None:
            _near(a[lo:hi], silu * u, (silu * u).abs() * _act_error(g), f"a {e}")


SPLITS = [
    [1],
    [0, 1, 0, 2, 0],
    [3, 0, 17, 1, 16, 15],
    [127, 128, 129, 0, 1],
    [255, 0, 256, 257, 63, 64, 65],
    [700, 5],
]
# (K, F): multiples of 8 and of nothing, around the tiles of 128 columns
WIDTHS = [(8, 8), (64, 128), (72, 40), (136, 264), (1000, 520), (1031, 517), (1, 1), (40, 129), (33, 64)]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("kf", WIDTHS)
@pytest.mark.parametrize("splits", SPLITS)
def test_both_directions(splits, kf, dtype):
    k, f = kf
    rows, g = sum(splits), len(splits)
    x, w = _normal((rows, k), 1, dtype), _normal((g, 2 * f, k), 2, dtype, k ** -0.5)
    h, a = mx.ragged_gemm_swiglu(x, w, _ms(splits))
    _check_forward(x, w, splits, None, h, a, rows)
    none, only = mx.ragged_gemm_swiglu(x, w, _ms(splits), want_h=False)
    assert none is None and torch.equal(only, a)
    dy, w2 = _normal((rows, k), 3, dtype), _normal((g, k, f), 4, dtype, k ** -0.5)
    dh, again = mx.ragged_gemm_swiglu_bwd(dy, w2, h, _ms(splits))
    _check_backward(dy, w2, h, splits, dh, again)
    alone, none = mx.ragged_gemm_swiglu_bwd(dy, w2, h, _ms(splits), want_a=False)
    assert none is None and torch.equal(alone, dh)


@pytest.mark.parametrize("rows_each,g,k,f", [
    (1, 3, 4096, 1040), (16, 8, 2048, 1024), (20, 4, 1024, 264),     # few rows
    (31, 8, 2304, 2048), (90, 4, 2304, 2048), (300, 3, 1024, 2048),  # tiles of 64, 128 and 256 rows
    (2000, 2, 512, 2560),                                            # more tiles than a round
])
def test_forms(rows_each, g, k, f):
    """Each form of the kernels, uneven experts; without a workspace nothing is split."""
    splits = [rows_each + (i % 3) - 1 for i in range(g)]
    rows = sum(splits)
    x, w = _normal((rows, k), 1, BF), _normal((g, 2 * f, k), 2, BF, k ** -0.5)
    h, a = mx.ragged_gemm_swiglu(x, w, _ms(splits))
    _check_forward(x, w, splits, None, h, a, rows)
    index = torch.randperm(rows, generator=torch.Generator().manual_seed(5)).int().cuda()
    h, a = mx.ragged_gemm_swiglu(x, w, _ms(splits), row_index=index)
    _check_forward(x, w, splits, index, h, a, rows)
    _, only = mx.ragged_gemm_swiglu(x, w, _ms(splits), row_index=index, want_h=False)
    assert torch.equal(only, a)
    w2 = _normal((g, k, f), 4, BF, k ** -0.5)
    dy = _normal((rows, k), 3, BF)
    dh, again = mx.ragged_gemm_swiglu_bwd(dy, w2, h, _ms(splits))
    _check_backward(dy, w2, h, splits, dh, again)


@pytest.mark.parametrize("kf", [(64, 128), (136, 264), (1031, 517)])
@pytest.mark.parametrize("tokens,splits", [(1, [1, 0, 1]), (40, [3, 0, 60, 17]), (300, [257, 0, 300, 343])])
def test_gather(tokens, splits, kf):
    """Any token any number of times; entries outside are rows of zeros."""
    k, f = kf
    rows, g = sum(splits), len(splits)
    index = torch.randint(0, tokens, (rows,), generator=torch.Generator().manual_seed(7)).int()
    if rows > 3:
        index[0], index[2], index[-1] = -1, tokens, 2 ** 31 - 1
    index = index.cuda()
    x, w = _normal((tokens, k), 1, BF), _normal((g, 2 * f, k), 2, BF, k ** -0.5)
    h, a = mx.ragged_gemm_swiglu(x, w, _ms(splits), row_index=index)
    _check_forward(x, w, splits, index, h, a, rows)
    if rows > 3:
        assert (a[0] == 0).all() and (h[2] == 0).all()


@pytest.mark.parametrize("kf", [(64, 128), (72, 40), (1031, 517)])
@pytest.mark.parametrize("rows,splits", [(150, [5, 3]), (150, [5, -4, 3]), (150, [100, 200, 30]), (150, [0, 0, 0]),
                                         (700, [300, 5]), (700, [900, 1])])
def test_splits_that_do_not_fill_the_rows(rows, splits, kf):
    """Rows behind the last expert are neither read nor written; long splits are cut."""
    k, f = kf
    g = len(splits)
    x, w = _normal((rows, k), 1, BF), _normal((g, 2 * f, k), 2, BF, k ** -0.5)
    dy, w2, hin = _normal((rows, k), 3, BF), _normal((g, k, f), 4, BF, k ** -0.5), _normal((rows, 2 * f), 5, BF)
    end = max(hi for _, hi in _spans(splits, rows))
    x[end:], dy[end:], hin[end:] = math.nan, math.inf, math.nan
    full = lambda c: torch.full((rows, c), 7.0, dtype=BF, device="cuda")  # noqa: E731
    h, a, dh, again = full(2 * f), full(f), full(2 * f), full(f)
    mx.ragged_gemm_swiglu(x, w, _ms(splits), h=h, out=a)
    _check_forward(x, w, splits, None, h, a, rows)
    mx.ragged_gemm_swiglu_bwd(dy, w2, hin, _ms(splits), dh=dh, out=again)
    _check_backward(dy, w2, hin, splits, dh, again)
    for t in (h, a, dh, again):
        assert (t[end:] == 7.0).all()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("k,f", [(1032, 2056), (2056, 3000)])   # one round of tiles; one and a part that is split
def test_high_tiles(k, f, dtype):
    """Tiles of 256 rows, gathered and not, both projections kept and not; experts that end inside one."""
    splits = [700, 5, 0, 1300, 257]
    rows, g, tokens = sum(splits), len(splits), 900
    index = torch.randint(-1, tokens + 1, (rows,), generator=torch.Generator().manual_seed(9)).int().cuda()
    w = _normal((g, 2 * f, k), 2, dtype, k ** -0.5)
    for x, at in ((_normal((rows, k), 1, dtype), None), (_normal((tokens, k), 3, dtype), index)):
        h, a = mx.ragged_gemm_swiglu(x, w, _ms(splits), row_index=at)
        _check_forward(x, w, splits, at, h, a, rows)
        none, only = mx.ragged_gemm_swiglu(x, w, _ms(splits), row_index=at, want_h=False)
        assert none is None and torch.equal(only, a)


@pytest.mark.parametrize("k,f", [(64, 128), (264, 136)])
@pytest.mark.parametrize("rows", [40, 600])
def test_strides_and_alignment(rows, k, f):
    """Strided and shifted operands and outputs give what contiguous ones give, within
    the order of sums; what lies between the rows stays."""
    splits = [rows - 7, 7]
    x, w = _normal((rows, k), 1, BF), _normal((2, 2 * f, k), 2, BF, k ** -0.5)
    for pad, shift in ((8, 0), (3, 0), (0, 1), (8, 5)):
        wide = torch.full((rows * (k + pad) + shift,), math.nan, dtype=BF, device="cuda")
        xs = wide[shift:].view(rows, k + pad)[:, :k]
        xs.copy_(x)
        buf = torch.full((rows * (f + pad) + shift,), 7.0, dtype=BF, device="cuda")
        out = buf[shift:].view(rows, f + pad)[:, :f]
        h, a = mx.ragged_gemm_swiglu(xs, w, _ms(splits), out=out)
        assert a is out
        _check_forward(x, w, splits, None, h, out, rows)
        assert (buf[:shift] == 7.0).all()
        assert (buf[shift:].view(rows, f + pad)[:, f:] == 7.0).all()
        dy = xs
        w2 = _normal((2, k, f), 4, BF, k ** -0.5)
        hs = torch.empty(rows * 2 * f + shift, dtype=BF, device="cuda")[shift:].view(rows, 2 * f)
        hs.copy_(h)
        dh, again = mx.ragged_gemm_swiglu_bwd(dy, w2, hs, _ms(splits))
        _check_backward(x, w2, h, splits, dh, again)


@pytest.mark.parametrize("rows", [5, 600])
def test_extreme_projections(rows):
    """Gates far from zero: the activation goes to 0 or the gate itself, nothing turns NaN;
    other experts' infinities reach no result."""
    k = f = 64
    x = torch.ones((rows, k), dtype=BF, device="cuda")
    w = torch.zeros((2, 2 * f, k), dtype=BF, device="cuda")
    gates = torch.tensor([-1e4, -200.0, -100.0, -88.0, -20.0, 0.0, 20.0, 88.0, 200.0, 1e4], device="cuda")
    w[0, :10, 0] = gates.to(BF)
    w[0, f:, 0] = 2.0
    w[1] = math.inf
    h, a = mx.ragged_gemm_swiglu(x, w, _ms([rows, 0]))
    g = w[0, :10, 0].double()
    want = torch.where(g < -700, 0.0, g * torch.sigmoid(g) * 2)
    _near(a[:, :10], want.expand(rows, 10), want.abs() * _act_error(g), "a")
    dy = torch.ones((rows, k), dtype=BF, device="cuda")
    w2 = torch.zeros((2, k, f), dtype=BF, device="cuda")
    w2[0, 0] = 1.0
    w2[1] = math.nan
    dh, again = mx.ragged_gemm_swiglu_bwd(dy, w2, h, _ms([rows, 0]))
    _check_backward(dy, w2[:1], h, [rows], dh, again)
    assert torch.equal(again, a)


def test_gradients_against_differences():
    """The chain forward, backward against central differences of the loss <a W2^T, d>."""
    torch.manual_seed(3)
    g, k, f, n, splits = 2, 24, 16, 32, [9, 4]
    x, w1, w2 = _normal((13, k), 1, BF), _normal((g, 2 * f, k), 2, BF, 0.4), _normal((g, n, f), 3, BF, 0.4)
    dy = _normal((13, n), 4, BF)
    expert = torch.tensor([0] * 9 + [1] * 4, device="cuda")

    def loss(x, w1, w2):
        z = torch.matmul(w1[expert], x[:, :, None])[:, :, 0]
        y = torch.matmul(w2[expert], (z[:, :f] * torch.sigmoid(z[:, :f]) * z[:, f:])[:, :, None])[:, :, 0]
        return (y * dy.double()).sum()

    h, _ = mx.ragged_gemm_swiglu(x, w1, _ms(splits))
    dh, a = mx.ragged_gemm_swiglu_bwd(dy, w2, h, _ms(splits))
    f32 = torch.float32
    got = {"x": mx.ragged_gemm("NN", dh, w1, _ms(splits), out_dtype=f32),
           "w1": mx.ragged_gemm("TN", dh, x, _ms(splits), out_dtype=f32),
           "w2": mx.ragged_gemm("TN", dy, a, _ms(splits), out_dtype=f32)}
    at = {"x": x.double(), "w1": w1.double(), "w2": w2.double()}
    big = torch.matmul(dy.double().abs()[:, None], w2.double().abs()[expert])[:, 0]      # of da
    both = torch.cat([1.1 * big * h[:, f:].double().abs(), big * h[:, :f].double().abs()], 1)
    of = torch.nn.functional.one_hot(expert, g).double().T[:, :, None]                   # rows of each expert
    per = lambda a, b: torch.matmul((of * a).transpose(1, 2).contiguous(), b.double().abs())  # noqa: E731
    sizes = {"x": torch.matmul(both[:, None], w1.double().abs()[expert])[:, 0], "w1": per(both, x),
             "w2": per(dy.double().abs(), (h[:, :f].double() * h[:, f:].double()).abs())}
    for name in at:
        for seed in range(4):
            step = torch.randn(at[name].shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda",
                               dtype=torch.float64)
            lo, hi = dict(at), dict(at)
            lo[name], hi[name] = at[name] - 1e-5 * step, at[name] + 1e-5 * step
            slope = float(loss(**hi) - loss(**lo)) / 2e-5
            # h, dh and a are rounded to bf16 once each, by at most 2^-8 of their size: three
            # roundings on any path, relative to the products of all factors' sizes
            off = 3 * 2.0 ** -8 * float((sizes[name] * step.abs()).sum())
            assert abs(float((got[name].double() * step).sum()) - slope) <= off, name


def test_no_rows_and_reused_buffers():
    x, w = _normal((0, 64), 1, BF), _normal((2, 256, 64), 2, BF)
    h, a = mx.ragged_gemm_swiglu(x, w, _ms([0, 0]))
    assert h.shape == (0, 256) and a.shape == (0, 128)
    dh, a = mx.ragged_gemm_swiglu_bwd(_normal((0, 64), 1, BF), _normal((2, 64, 128), 2, BF), h, _ms([0, 0]))
    assert dh.shape == (0, 256) and a.shape == (0, 128)
    # rows, but of no token: all rows of zeros
    index = torch.zeros(3, dtype=torch.int32, device="cuda")
    h, a = mx.ragged_gemm_swiglu(x, w, _ms([2, 1]), row_index=index)
    assert (h == 0).all() and (a == 0).all()


def test_captured_and_replayed():
    """Both calls in one graph with a workspace of their own, replayed on new inputs with
    eager work between."""
    splits, k, f = [300, 0, 420, 100], 512, 384
    rows = sum(splits)
    ms = _ms(splits)
    x, w, w2 = _normal((rows, k), 1, BF), _normal((4, 2 * f, k), 2, BF, 0.05), _normal((4, k, f), 3, BF, 0.05)
    dy = _normal((rows, k), 4, BF)
    need = max(mx.ragged_gemm_swiglu_workspace_bytes(b, rows, f, k, 4) for b in (False, True))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    bufs = dict(h=torch.empty((rows, 2 * f), dtype=BF, device="cuda"), out=torch.empty((rows, f), dtype=BF, device="cuda"))
    back = dict(dh=torch.empty((rows, 2 * f), dtype=BF, device="cuda"), out=torch.empty((rows, f), dtype=BF, device="cuda"))

    def step():
        mx.ragged_gemm_swiglu(x, w, ms, workspace=ws, **bufs)
        mx.ragged_gemm_swiglu_bwd(dy, w2, bufs["h"], ms, workspace=ws, **back)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        x.copy_(_normal((rows, k), 10 + seed, BF))
        dy.copy_(_normal((rows, k), 20 + seed, BF))
        graph.replay()
        got = [t.clone() for t in (*bufs.values(), *back.values())]
        h, a = mx.ragged_gemm_swiglu(x, w, ms)
        dh, again = mx.ragged_gemm_swiglu_bwd(dy, w2, h, ms)
        torch.cuda.synchronize()
        for one, other in zip(got, (h, a, dh, again)):
            assert torch.equal(one, other)


@pytest.mark.parametrize("splits,k,f", [([300, 0, 65, 128], 1031, 517), ([1300, 0, 1665, 1128], 257, 1031)])
def test_any_size_tiles(splits, k, f):
    """The any-size form with tiles of 64 and of 128 rows, both directions."""
    rows, g = sum(splits), len(splits)
    x, w = _normal((rows, k), 1, BF), _normal((g, 2 * f, k), 2, BF, k ** -0.5)
    index = torch.randint(-1, rows + 1, (rows,), generator=torch.Generator().manual_seed(4)).int().cuda()
    h, a = mx.ragged_gemm_swiglu(x, w, _ms(splits), row_index=index)
    _check_forward(x, w, splits, index, h, a, rows)
    dy, w2 = _normal((rows, k), 3, BF), _normal((g, k, f), 4, BF, k ** -0.5)
    _check_backward(dy, w2, h, splits, *mx.ragged_gemm_swiglu_bwd(dy, w2, h, _ms(splits)))
