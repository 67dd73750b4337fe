"""Products grouped by expert with ragged row counts (bf16, fp16 and 8-bit
integers) against plain per-expert products in float64."""

import math

import pytest
import torch

import moe_expert_grouped_group_amd as mx

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def _normal(shape, seed, dtype, std=1.0):
    gen = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").mul_(std).to(dtype)


def _spans(splits, rows):
    """[lo, hi) of each expert as the operator defines it."""
    lo, got = 0, []
    for m in splits:
        hi = min(lo + max(m, 0), rows)
        got.append((min(lo, rows), hi))
        lo += max(m, 0)
    return got


def _gather(x, index):
    """Rows of x in float64; entries outside the rows give zeros."""
    if index is None:
        return x.double()
    at = index.long()
    ok = (at >= 0) & (at < x.shape[0])
    if x.shape[0] == 0:
        return torch.zeros((at.numel(), x.shape[1]), dtype=torch.float64, device=x.device)
    return torch.where(ok[:, None], x[at.clamp(0, x.shape[0] - 1)].double(), 0.0)


def _check(got, ref, mag, terms, what=""):
    """Products of 16-bit values are exact in fp32; a sum of `terms` of them is
    formed in steps of at most 16 terms, each addition off by at most one fp32
    step of the magnitude summed so far; then one rounding to the output type."""
    step = terms / 16 + 20
    tol = mag * step * 2.0 ** -23 + ref.abs() * torch.finfo(got.dtype).eps / 2
    tol = tol + torch.finfo(got.dtype).smallest_normal
    off = (got.double() - ref).abs()
    assert not torch.isnan(got).any(), what
    bad = off > tol
    assert not bad.any(), (what, int(bad.sum()), float((off / tol).max()))


def _forward(x, w, splits, index, got, rows):
    for g, (lo, hi) in enumerate(_spans(splits, rows)):
        a = _gather(x, index)[lo:hi]
        b = w[g].double()
        _check(got[lo:hi], a @ b.T, a.abs() @ b.abs().T, x.shape[1], f"expert {g}")


def _dgrad(dy, w, splits, got):
    for g, (lo, hi) in enumerate(_spans(splits, dy.shape[0])):
        a, b = dy[lo:hi].double(), w[g].double()
        _check(got[lo:hi], a @ b, a.abs() @ b.abs(), dy.shape[1], f"expert {g}")


def _wgrad(dy, x, splits, index, got):
    for g, (lo, hi) in enumerate(_spans(splits, dy.shape[0])):
        a, b = dy[lo:hi].double(), _gather(x, index)[lo:hi]
        if hi == lo:
            assert (got[g] == 0).all(), f"expert {g}"
        else:
            _check(got[g], a.T @ b, a.abs().T @ b.abs(), hi - lo, f"expert {g}")


def _ms(splits):
    return torch.tensor(splits, dtype=torch.int64, device="cuda")


# rows around the tile edges, experts without rows at both ends and between
SPLITS = [
    [1],
    [0, 1, 0, 2, 0],
    [3, 0, 17, 1, 16, 15],
    [127, 128, 129, 0, 1],
    [255, 0, 256, 257, 63, 64, 65],
    [700, 5],
]
# (K, N): multiples of 8 and of nothing, shorter and longer than a tile
WIDTHS = [(8, 8), (64, 256), (72, 40), (136, 264), (512, 520), (1000, 1031), (1031, 517), (1, 1)]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("kn", WIDTHS)
@pytest.mark.parametrize("splits", SPLITS)
def test_products(splits, kn, dtype):
    k, n = kn
    rows, g = sum(splits), len(splits)
    ms = _ms(splits)
    x = _normal((rows, k), 1, dtype)
    w = _normal((g, n, k), 2, dtype)
    dy = _normal((rows, n), 3, dtype)
    for out in (dtype, F32):
        _forward(x, w, splits, None, mx.ragged_gemm("NT", x, w, ms, out_dtype=out), rows)
        _dgrad(dy, w, splits, mx.ragged_gemm("NN", dy, w, ms, out_dtype=out))
        _wgrad(dy, x, splits, None, mx.ragged_gemm("TN", dy, x, ms, out_dtype=out))


@pytest.mark.parametrize("kn", [(64, 256), (136, 264), (1031, 517)])
@pytest.mark.parametrize("tokens,splits", [(1, [1, 0, 1]), (40, [3, 0, 60, 17]),
                                           (300, [257, 0, 300, 43])])
def test_gather(tokens, splits, kn):
    """row_index: any token any number of times; entries outside are rows of zeros."""
    k, n = kn
    rows, g = sum(splits), len(splits)
    gen = torch.Generator().manual_seed(7)
    index = torch.randint(0, tokens, (rows,), generator=gen).to(torch.int32).cuda()
    if rows > 3:
        index[0], index[2] = -1, tokens
    x, w, dy = _normal((tokens, k), 1, BF), _normal((g, n, k), 2, BF), _normal((rows, n), 3, BF)
    got = mx.ragged_gemm("NT", x, w, _ms(splits), row_index=index)
    _forward(x, w, splits, index, got, rows)
    _wgrad(dy, x, splits, index, mx.ragged_gemm("TN", dy, x, _ms(splits), row_index=index))


@pytest.mark.parametrize("kn", [(64, 256), (72, 40), (136, 264), (1031, 517)])
@pytest.mark.parametrize("splits", [[5, 3], [5, -4, 3], [100, 200, 30], [0, 0, 0], [300, 0, 1]])
def test_splits_that_do_not_fill_the_rows(splits, kn):
    """Sums short of the rows leave the rest untouched and unread; longer ones
    are cut; negative ones count as empty."""
    k, n = kn
    rows, g = 150, len(splits)
    x, w, dy = _normal((rows, k), 1, BF), _normal((g, n, k), 2, BF), _normal((rows, n), 3, BF)
    end = max(hi for _, hi in _spans(splits, rows))
    x[end:], dy[end:] = math.nan, math.inf
    index = torch.arange(rows, dtype=torch.int32, device="cuda")
    for idx in (None, index):
        out = torch.full((rows, n), 7.0, dtype=BF, device="cuda")
        mx.ragged_gemm("NT", x, w, _ms(splits), row_index=idx, out=out)
        _forward(x, w, splits, idx, out, rows)
        assert (out[end:] == 7.0).all()
        _wgrad(dy, x, splits, idx, mx.ragged_gemm("TN", dy, x, _ms(splits), row_index=idx))
    out = torch.full((rows, k), 7.0, dtype=BF, device="cuda")
    mx.ragged_gemm("NN", dy, w, _ms(splits), out=out)
    _dgrad(dy, w, splits, out)
    assert (out[end:] == 7.0).all()


@pytest.mark.parametrize("kn", [(64, 72), (72, 264), (1031, 517)])
def test_values_of_other_rows_stay_out(kn):
    """An expert whose rows hold NaN, and weights that hold infinities, spoil
    their own results only."""
    k, n = kn
    splits = [5, 70, 130, 0, 3]
    rows = sum(splits)
    x, w, dy = _normal((rows, k), 1, BF), _normal((5, n, k), 2, BF), _normal((rows, n), 3, BF)
    x[5:75], dy[5:75] = math.nan, math.nan
    w[1] = math.inf
    y = mx.ragged_gemm("NT", x, w, _ms(splits))
    dx = mx.ragged_gemm("NN", dy, w, _ms(splits))
    dw = mx.ragged_gemm("TN", dy, x, _ms(splits))
    assert torch.isnan(y[5:75]).all() and torch.isnan(dx[5:75]).all() and torch.isnan(dw[1]).all()
    for g, (lo, hi) in enumerate(_spans(splits, rows)):
        if g != 1:
            a, b, d = x[lo:hi].double(), w[g].double(), dy[lo:hi].double()
            _check(y[lo:hi], a @ b.T, a.abs() @ b.abs().T, k)
            _check(dx[lo:hi], d @ b, d.abs() @ b.abs(), n)
            _check(dw[g], d.T @ a, d.abs().T @ a.abs(), max(hi - lo, 1))


@pytest.mark.parametrize("shift", [0, 1, 8])
@pytest.mark.parametrize("kn,pad", [((64, 256), 8), ((64, 256), 3), ((136, 264), 8), ((37, 50), 5)])
def test_strides_and_alignment(kn, pad, shift):
    """Row strides longer than a row, pointers off 16 bytes, and a frame around
    every output that stays as it was."""
    k, n = kn
    splits = [3, 90, 0, 260]
    rows = sum(splits)

    def strided(t):
        flat = torch.full((t.shape[0] * (t.shape[1] + pad) + shift + pad,), math.nan, dtype=t.dtype,
                          device="cuda")
        v = flat[shift:shift + t.shape[0] * (t.shape[1] + pad)].view(t.shape[0], -1)[:, :t.shape[1]]
        v.copy_(t)
        return flat, v

    _, x = strided(_normal((rows, k), 1, HF))
    _, dy = strided(_normal((rows, n), 3, HF))
    wf = torch.full((4 * n * k + shift,), math.nan, dtype=HF, device="cuda")
    w = wf[shift:].view(4, n, k)
    w.copy_(_normal((4, n, k), 2, HF))
    for layout, a, b, cols in (("NT", x, w, n), ("NN", dy, w, k)):
        flat, out = strided(torch.zeros((rows, cols), dtype=HF, device="cuda"))
        mx.ragged_gemm(layout, a, b, _ms(splits), out=out)
        if layout == "NT":
            _forward(x, w, splits, None, out, rows)
        else:
            _dgrad(dy, w, splits, out)
        out.fill_(math.nan)
        assert torch.isnan(flat).all()
    flat = torch.full((4 * n * k + 64,), 7.0, dtype=F32, device="cuda")
    out = flat[32:32 + 4 * n * k].view(4, n, k)
    mx.ragged_gemm("TN", dy, x, _ms(splits), out_dtype=F32, out=out)
    _wgrad(dy, x, splits, None, out)
    assert (flat[:32] == 7.0).all() and (flat[32 + 4 * n * k:] == 7.0).all()


@pytest.mark.parametrize("rows,k,n,g", [(64, 4096, 512, 1), (777, 2048, 776, 3), (2500, 520, 1288, 2),
                                        (16, 4096, 1000, 8), (40, 1288, 256, 20), (3, 8192, 96, 2)])
def test_whole_numbers_are_exact(rows, k, n, g):
    """Small whole numbers: every sum is exact in fp32, so the results are equal."""
    gen = torch.Generator("cuda").manual_seed(5)
    draw = lambda *s: torch.randint(-4, 5, s, generator=gen, device="cuda")  # noqa: E731
    cut = sorted(torch.randint(0, rows + 1, (g - 1,), generator=torch.Generator().manual_seed(3)).tolist())
    splits = [b - a for a, b in zip([0] + cut, cut + [rows])]
    x, w, dy = draw(rows, k).to(BF), draw(g, n, k).to(BF), draw(rows, n).to(BF)
    y = mx.ragged_gemm("NT", x, w, _ms(splits), out_dtype=F32)
    dx = mx.ragged_gemm("NN", dy, w, _ms(splits), out_dtype=F32)
    dw = mx.ragged_gemm("TN", dy, x, _ms(splits), out_dtype=F32)
    for i, (lo, hi) in enumerate(_spans(splits, rows)):
        assert torch.equal(y[lo:hi].double(), x[lo:hi].double() @ w[i].double().T)
        assert torch.equal(dx[lo:hi].double(), dy[lo:hi].double() @ w[i].double())
        assert torch.equal(dw[i].double(), dy[lo:hi].double().T @ x[lo:hi].double())


def test_gradients_against_differences():
    """The three products are the derivative of <C, D>: along random directions
    of X and W the change of the loss equals the gradients' inner products (the
    loss is linear in each, so differences are exact up to rounding)."""
    splits, k, n = [3, 0, 21, 9], 24, 40
    rows = sum(splits)
    x, w, d = _normal((rows, k), 1, BF), _normal((4, n, k), 2, BF), _normal((rows, n), 3, BF)
    ms = _ms(splits)
    dx = mx.ragged_gemm("NN", d, w, ms, out_dtype=F32).double()
    dw = mx.ragged_gemm("TN", d, x, ms, out_dtype=F32).double()
    loss = lambda a, b: (mx.ragged_gemm("NT", a, b, ms, out_dtype=F32).double() * d.double()).sum()  # noqa: E731
    for seed in range(3):
        # steps on bf16's grid at twice the scale, so that x + step is exact
        ex = (x * 2 ** torch.randint(0, 2, x.shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(BF))
        ew = (w * 2 ** torch.randint(0, 2, w.shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(BF))
        # |loss| terms: rows * n sums of k products; fp32 steps of each
        scale = float((d.double().abs() * 1.0).sum()) * k * 64 * 2.0 ** -23
        assert abs(float(loss(ex, w) - loss(x, w) - ((ex.double() - x.double()) * dx).sum())) < scale
        assert abs(float(loss(x, ew) - loss(x, w) - ((ew.double() - w.double()) * dw).sum())) < scale


def test_same_from_run_to_run_and_on_another_stream():
    splits, k, n = [9, 300, 0, 41], 520, 264
    x, w = _normal((350, k), 1, BF), _normal((4, n, k), 2, BF)
    dy = _normal((350, n), 3, BF)
    ms = _ms(splits)
    first = [mx.ragged_gemm("NT", x, w, ms), mx.ragged_gemm("NN", dy, w, ms),
             mx.ragged_gemm("TN", dy, x, ms)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = [mx.ragged_gemm("NT", x, w, ms, stream=s), mx.ragged_gemm("NN", dy, w, ms, stream=s),
             mx.ragged_gemm("TN", dy, x, ms, stream=s)]
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(first, again):
        assert torch.equal(a, b)


def test_graph_replays_follow_new_inputs():
    k, n = 136, 72
    x, w = _normal((200, k), 1, BF), _normal((3, n, k), 2, BF)
    dy = _normal((200, n), 3, BF)
    ms = _ms([50, 100, 50])
    q, sc = mx.quantize_int8(x)
    wq, ws = mx.quantize_int8(w.view(3 * n, k))
    wq, ws = wq.view(3, n, k), ws.view(3, n)
    outs = [torch.empty((200, n), dtype=BF, device="cuda"), torch.empty((200, k), dtype=BF, device="cuda"),
            torch.empty((3, n, k), dtype=BF, device="cuda"), torch.empty((200, n), dtype=BF, device="cuda")]

    def step():
        mx.ragged_gemm("NT", x, w, ms, out=outs[0])
        mx.ragged_gemm("NN", dy, w, ms, out=outs[1])
        mx.ragged_gemm("TN", dy, x, ms, out=outs[2])
        mx.quantize_int8(x, out=(q, sc))
        mx.ragged_gemm_int8(q, sc, wq, ws, ms, out=outs[3])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i, splits in enumerate(([50, 100, 50], [0, 200, 0], [199, 0, 1], [66, 67, 67])):
        ms.copy_(_ms(splits))
        x.copy_(_normal((200, k), 10 + i, BF))
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, outs):
            assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# 8-bit integers
# ---------------------------------------------------------------------------

def _codes(x):
    """Scale and codes by definition, in float64 on the CPU."""
    v = x.double().cpu()
    scale = (v.abs().amax(1) / 127).float()
    codes = torch.where(scale[:, None] > 0, torch.round(v / scale.double()[:, None]), 0.0)
    return codes, scale


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("t,k", [(1, 1), (3, 7), (5, 8), (17, 1000), (4, 8192), (3, 8199), (2, 20001)])
def test_quantize(t, k, dtype):
    x = _normal((t, k), 1, dtype)
    x[0, :] *= 1e-3
    q, s = mx.quantize_int8(x)
    codes, scale = _codes(x)
    assert torch.equal(s.cpu(), scale)
    assert torch.equal(q.cpu().double(), codes)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_quantize_ties_extremes_and_edges(dtype):
    """Quotients on the border between two integers go to the even one; zeros,
    the smallest and largest numbers; infinities and NaN give scale NaN."""
    fi = torch.finfo(dtype)
    rows = [torch.arange(-127, 128, dtype=torch.float64)[:254] / 2,             # amax 63.5: x / s = 2 x
            (torch.arange(254, dtype=torch.float64) - 127) + 0.0,
            torch.full((254,), 0.0),
            torch.linspace(-1, 1, 254, dtype=torch.float64) * float(fi.max),
            torch.linspace(-1, 1, 254, dtype=torch.float64) * float(fi.smallest_normal),
            torch.linspace(-8, 8, 254, dtype=torch.float64) * float(fi.smallest_normal) * fi.eps]
    # halves against a power-of-two scale: 127 s with s = 2^-3, ties at odd multiples of s / 2
    tie = torch.cat([torch.tensor([127 / 8]), (torch.arange(253, dtype=torch.float64) - 126) / 16])
    x = torch.stack([r.double() for r in rows] + [tie]).to(dtype).cuda()
    q, s = mx.quantize_int8(x)
    codes, scale = _codes(x)
    assert torch.equal(s.cpu(), scale)
    assert torch.equal(q.cpu().double(), codes)
    assert s[2] == 0 and (q[2] == 0).all()
    for bad in (math.inf, -math.inf, math.nan):
        y = _normal((2, 100), 1, dtype)
        y[1, 77] = bad
        q, s = mx.quantize_int8(y)
        assert torch.isnan(s[1]) and (q[1] == 0).all() and torch.isfinite(s[0])


def test_quantize_strided():
    big = _normal((9, 300), 1, BF)
    for lo in (0, 1, 8):
        q, s = mx.quantize_int8(big[:, lo:lo + 250])
        codes, scale = _codes(big[:, lo:lo + 250])
        assert torch.equal(s.cpu(), scale) and torch.equal(q.cpu().double(), codes)


def _int8_check(q, sc, w, ws, splits, index, got, rows):
    """The integer sum is exact; then a conversion to fp32, two products and the
    output's rounding, half a step each (the first three of fp32)."""
    a = _gather(q, index)
    s = _gather(sc[:, None], index)[:, 0]
    for g, (lo, hi) in enumerate(_spans(splits, rows)):
        ref = (a[lo:hi] @ w[g].double().T) * s[lo:hi, None] * ws[g].double()
        tol = ref.abs() * (3.01 * 2.0 ** -24 + torch.finfo(got.dtype).eps / 2)
        tol = tol + torch.finfo(got.dtype).smallest_normal
        off = (got[lo:hi].double() - ref).abs()
        assert (off <= tol).all(), f"expert {g}: {float((off / tol).max())}"


@pytest.mark.parametrize("out", [F32, BF, HF])
@pytest.mark.parametrize("kn", [(16, 16), (128, 256), (144, 40), (1000, 1031), (1031, 517), (1, 1)])
@pytest.mark.parametrize("splits", SPLITS)
def test_int8(splits, kn, out):
    k, n = kn
    rows, g = sum(splits), len(splits)
    gen = torch.Generator("cuda").manual_seed(1)
    q = torch.randint(-127, 128, (rows, k), generator=gen, device="cuda", dtype=torch.int8)
    w = torch.randint(-127, 128, (g, n, k), generator=gen, device="cuda", dtype=torch.int8)
    sc, ws = torch.rand(rows, generator=gen, device="cuda") * 1e-2, torch.rand((g, n), generator=gen, device="cuda") * 1e-2
    got = mx.ragged_gemm_int8(q, sc, w, ws, _ms(splits), out_dtype=out)
    _int8_check(q, sc, w, ws, splits, None, got, rows)


@pytest.mark.parametrize("kn", [(128, 256), (1040, 264), (1031, 517)])
@pytest.mark.parametrize("tokens,splits", [(1, [1, 0, 1]), (40, [3, 0, 60, 17]), (300, [257, 0, 300, 43])])
def test_int8_gather_and_short_splits(tokens, splits, kn):
    k, n = kn
    rows, g = sum(splits) + 5, len(splits)
    gen = torch.Generator("cuda").manual_seed(2)
    q = torch.randint(-128, 128, (tokens, k), generator=gen, device="cuda", dtype=torch.int8)
    w = torch.randint(-128, 128, (g, n, k), generator=gen, device="cuda", dtype=torch.int8)
    sc, ws = torch.rand(tokens, generator=gen, device="cuda"), torch.rand((g, n), generator=gen, device="cuda")
    index = torch.randint(0, tokens, (rows,), generator=gen, device="cuda").int()
    index[-5:] = -1
    if rows > 8:
        index[0], index[2] = -1, tokens
    out = torch.full((rows, n), 7.0, dtype=F32, device="cuda")
    mx.ragged_gemm_int8(q, sc, w, ws, _ms(splits), row_index=index, out_dtype=F32, out=out)
    _int8_check(q, sc, w, ws, splits, index, out, rows)
    assert (out[-5:] == 7.0).all()


def test_int8_longest_sum():
    """K = 131071 of the largest products stays within 32 bits."""
    k = 131071
    q = torch.full((2, k), 127, dtype=torch.int8, device="cuda")
    w = torch.full((1, 3, k), -128, dtype=torch.int8, device="cuda")
    got = mx.ragged_gemm_int8(q, torch.ones(2, device="cuda"), w, torch.ones((1, 3), device="cuda"),
                              _ms([2]), out_dtype=F32)
    assert (got.double() + 127.0 * 128 * k).abs().max() <= 127 * 128 * k * 2.0 ** -24


# Weights so large that few rows do not pay for the forward form of few rows:
# the large tiles of 64, 128 and 256 rows.  (K, N): contractions that end inside
# a 16-byte chunk's stage, are one stage or less, columns that end inside a tile.
TILED = [(6152, 4104, [20, 0, 41, 1, 64, 33]), (6208, 4136, [63, 65, 0, 130, 100, 1]),
         (6144, 4104, [300, 257, 0, 1, 255, 256]), (72, 300008, [30, 64, 0, 40]),
         (136, 160040, [129, 128, 0, 127]), (8, 1000008, [70, 80]), (64, 260040, [200, 0, 150, 1])]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("k,n,splits", TILED)
def test_forward_large_tiles(k, n, splits, gather):
    rows, g = sum(splits), len(splits)
    x, w = _normal((rows, k), 1, BF), _normal((g, n, k), 2, BF)
    index = None
    if gather:
        index = torch.randperm(rows, generator=torch.Generator().manual_seed(3)).int().cuda()
        index[0], index[5] = -1, rows
    _forward(x, w, splits, index, mx.ragged_gemm("NT", x, w, _ms(splits), row_index=index), rows)
    if k > 64:
        got = mx.ragged_gemm("NT", x, w, _ms(splits), row_index=index, out_dtype=F32)
        _forward(x, w, splits, index, got, rows)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("k,n,splits", [(12304, 4104, [20, 0, 41, 1, 64, 33]), (12416, 4136, [63, 65, 0, 130, 100, 1]),
                                        (12288, 4104, [300, 257, 0, 1, 255, 256]), (144, 300016, [30, 64, 0, 40]),
                                        (272, 160048, [129, 128, 0, 127]), (16, 1000016, [70, 80])])
def test_int8_large_tiles(k, n, splits, gather):
    rows, g = sum(splits), len(splits)
    gen = torch.Generator("cuda").manual_seed(2)
    q = torch.randint(-127, 128, (rows, k), generator=gen, device="cuda", dtype=torch.int8)
    w = torch.randint(-127, 128, (g, n, k), generator=gen, device="cuda", dtype=torch.int8)
    sc, ws = torch.rand(rows, generator=gen, device="cuda"), torch.rand((g, n), generator=gen, device="cuda")
    index = None
    if gather:
        index = torch.randperm(rows, generator=torch.Generator().manual_seed(3)).int().cuda()
        index[0], index[5] = -1, rows
    got = mx.ragged_gemm_int8(q, sc, w, ws, _ms(splits), row_index=index, out_dtype=BF)
    _int8_check(q, sc, w, ws, splits, index, got, rows)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("k,n,pad", [(2111, 4011, 0), (2112, 4011, 3), (2111, 4008, 5)])
def test_odd_operands_laid_out_anew(k, n, pad, dtype):
    """Rows that do not start on 16 bytes, and work enough that they are copied
    first; rows past the last expert's are neither read nor written."""
    splits, rows = [1200, 0, 1, 900, 850], 3000
    g, end = len(splits), sum(splits)
    wide = lambda t: torch.nn.functional.pad(t, (0, pad), value=math.nan)[:, :t.shape[1]]  # noqa: E731
    x, dy = _normal((rows, k), 1, dtype), _normal((rows, n), 3, dtype)
    x[end:], dy[end:] = math.nan, math.inf
    x, dy, w, ms = wide(x), wide(dy), _normal((g, n, k), 2, dtype), _ms(splits)
    index = torch.arange(rows - 1, -1, -1, dtype=torch.int32, device="cuda")
    xr = x.flip(0).contiguous()          # the same rows through the index
    for out in (dtype, F32):
        y = wide(torch.full((rows, n), 7.0, dtype=out, device="cuda"))
        mx.ragged_gemm("NT", x, w, ms, out=y, out_dtype=out)
        _forward(x, w, splits, None, y, rows)
        assert (y[end:] == 7.0).all()
        y2 = mx.ragged_gemm("NT", xr, w, ms, row_index=index, out_dtype=out)
        assert torch.equal(y2[:end], y[:end])
        dx = torch.full((rows, k), 7.0, dtype=out, device="cuda")
        mx.ragged_gemm("NN", dy, w, ms, out=dx, out_dtype=out)
        _dgrad(dy, w, splits, dx)
        assert (dx[end:] == 7.0).all()
        dw = mx.ragged_gemm("TN", dy, x, ms, out_dtype=out)
        _wgrad(dy, x, splits, None, dw)
        assert torch.equal(mx.ragged_gemm("TN", dy, xr, ms, row_index=index, out_dtype=out), dw)


def test_int8_odd_laid_out_anew():
    splits, k, n, rows = [1200, 0, 1, 900, 850], 2111, 4011, 3000
    gen = torch.Generator("cuda").manual_seed(2)
    q = torch.randint(-127, 128, (rows, k), generator=gen, device="cuda", dtype=torch.int8)
    w = torch.randint(-127, 128, (5, n, k), generator=gen, device="cuda", dtype=torch.int8)
    sc, ws = torch.rand(rows, generator=gen, device="cuda"), torch.rand((5, n), generator=gen, device="cuda")
    for out in (F32, BF, HF):
        _int8_check(q, sc * 1e-3, w, ws * 1e-3, splits, None,
                    mx.ragged_gemm_int8(q, sc * 1e-3, w, ws * 1e-3, _ms(splits), out_dtype=out), rows)


def test_wgrad_odd_columns_of_padded_rows():
    """Odd widths in rows that do start on 16 bytes: the last value of the last row."""
    splits, k, n = [70, 0, 130], 37, 51
    x, dy = torch.zeros((200, 40), dtype=BF, device="cuda")[:, :k], torch.zeros((200, 56), dtype=BF, device="cuda")[:, :n]
    x.copy_(_normal((200, k), 1, BF))
    dy.copy_(_normal((200, n), 2, BF))
    _wgrad(dy, x, splits, None, mx.ragged_gemm("TN", dy, x, _ms(splits)))
    k = 40
    x = _normal((200, k), 1, BF)
    _wgrad(dy, x, splits, None, mx.ragged_gemm("TN", dy, x, _ms(splits), out_dtype=F32))


def test_small_workspace_and_none():
    """A workspace that is larger than needed, and the C entry without one."""
    from moe_expert_grouped_group_amd import _native
    splits, k, n = [300, 0, 700], 1032, 520
    x, w, dy, ms = _normal((1000, k), 1, BF), _normal((3, n, k), 2, BF), _normal((1000, n), 3, BF), _ms(splits)
    need = mx.ragged_gemm_workspace_bytes("NN", BF, 1000, 1000, n, k, 3)
    big = torch.empty(need + 4096, dtype=torch.uint8, device="cuda")
    a = mx.ragged_gemm("NN", dy, w, ms, out_dtype=F32, workspace=big)
    assert torch.equal(a, mx.ragged_gemm("NN", dy, w, ms, out_dtype=F32))
    with pytest.raises(ValueError):
        mx.ragged_gemm("NN", dy, w, ms, workspace=big[:need - 1])
    b = torch.empty_like(a)
    lib = _native.load()
    st = lib.mxfp8_ragged_gemm(1, 1, dy.data_ptr(), n, w.data_ptr(), k, b.data_ptr(), k, 0, 1000, 1000, n, k,
                               ms.data_ptr(), 3, None, None, 0, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    _dgrad(dy, w, splits, b)


def test_offsets_past_32_bits():
    """Weights, gathered tokens and outputs over 4 GiB."""
    g, n, k = 33, 8192, 8192                      # W: 4.4 GB
    w = torch.empty((g, n, k), dtype=BF, device="cuda")
    for i in range(g):
        w[i] = _normal((n, k), 100 + i, BF)
    splits = [0] * (g - 2) + [3, 300]
    x, dy = _normal((303, k), 1, BF), _normal((303, n), 3, BF)
    _forward(x, w, splits, None, mx.ragged_gemm("NT", x, w, _ms(splits)), 303)
    _dgrad(dy, w, splits, mx.ragged_gemm("NN", dy, w, _ms(splits)))
    del w
    tokens, k, n = 270000, 8200, 16               # X: 4.4 GB
    x = torch.zeros((tokens, k), dtype=BF, device="cuda")
    x[-500:] = _normal((500, k), 5, BF)
    w, dy = _normal((2, n, k), 2, BF), _normal((400, n), 3, BF)
    index = (tokens - 1 - torch.arange(400, device="cuda")).int()
    _forward(x, w, [150, 250], index, mx.ragged_gemm("NT", x, w, _ms([150, 250]), row_index=index), 400)
    _wgrad(dy, x, [150, 250], index, mx.ragged_gemm("TN", dy, x, _ms([150, 250]), row_index=index))
    # the same tensor as rows of the product, most of them one expert's
    got = mx.ragged_gemm("NT", x, w, _ms([tokens - 300, 300]))
    assert (got[:tokens - 500] == 0).all()
    tail = _normal((500, k), 5, BF)
    _forward(tail, w, [200, 300], None, got[-500:], 500)
    big = _normal((tokens, n), 9, BF)
    dw = mx.ragged_gemm("TN", big, x, _ms([tokens - 300, 300]), out_dtype=F32)
    _wgrad(big[-500:], tail, [200, 300], None, dw)
    del x
    out = mx.ragged_gemm("NN", big, w, _ms([tokens - 300, 300]))      # C: 4.4 GB
    _dgrad(big[-500:], w, [200, 300], out[-500:])
