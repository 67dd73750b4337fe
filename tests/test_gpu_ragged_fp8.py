"""8-bit floating point with a scale for each block of 128: the quantizers against the
definition in float64, the products grouped by expert against plain ones."""

import math

import pytest
import torch

import moe_expert_grouped_group_amd as mx

pytestmark = pytest.mark.gpu

BF, HF, F32, F8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


def _normal(shape, seed, dtype, std=1.0):
    gen = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").mul_(std).to(dtype)


def _ms(splits):
    return torch.tensor(splits, dtype=torch.int64, device="cuda")


def _blocks(n):
    return -(-n // 128)


def _spread(scale, shape):
    """Scales of blocks (the last two dimensions, or the last one) spread over their values."""
    s = scale.double().repeat_interleave(128, dim=-1)[..., :shape[-1]]
    if scale.dim() == 3:
        s = s.repeat_interleave(128, dim=-2)[..., :shape[-2], :]
    return s


# the finite e4m3 values from 0 up; the place in this list is the code
CODES = [m / 512 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1]


def _codes_of(x, scale):
    """The nearest code of x / scale (float64), ties to the even one; uint8."""
    codes = torch.tensor(CODES, dtype=torch.float64, device=x.device)
    v = (x.double() / torch.where(scale == 0, 1.0, scale)).abs()
    # both sides of a border times the scale, exact in float64 (5 + 24 and 11 bits): no division decides
    middle = (codes[1:] + codes[:-1]) / 2
    at = torch.searchsorted(middle, v)
    for step in (0, 1):                                  # mend what the division rounded
        low = torch.clamp(at - 1, min=0)
        at = torch.where((at > 0) & (x.double().abs() < middle[low] * scale), at - 1, at)
        up = torch.clamp(at, max=len(CODES) - 2)
        at = torch.where((at < len(CODES) - 1) & (x.double().abs() > middle[up] * scale), at + 1, at)
    up, low = torch.clamp(at, max=len(CODES) - 2), torch.clamp(at - 1, min=0)
    at = torch.where((at < len(CODES) - 1) & (x.double().abs() == middle[up] * scale) & (at % 2 == 1), at + 1, at)
    at = torch.where((at > 0) & (x.double().abs() == middle[low] * scale) & (at % 2 == 1), at - 1, at)
    return (at + 128 * torch.signbit(x).long()).to(torch.uint8)


def _check_codes(x, q, scale):
    """Equal to the last bit: every scale, and every code (that of a zero keeps its sign)."""
    shape = x.shape
    if scale.dim() == 2:
        wide = torch.nn.functional.pad(x.abs(), (0, -shape[-1] % 128)).view(shape[0], -1, 128).amax(2)
    else:
        wide = torch.nn.functional.pad(x.abs(), (0, -shape[-1] % 128, 0, -shape[-2] % 128))
        wide = wide.view(shape[0], _blocks(shape[1]), 128, -1, 128).amax((2, 4))
    assert torch.equal(scale, (wide.double() / 448).float())
    over = _spread(scale, shape)
    want = torch.where(over == 0, 0, _codes_of(x, over).int()).to(torch.uint8)
    got = q.view(torch.uint8)
    bad = got != want
    assert not bad.any(), (int(bad.sum()), x[bad][:4], got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("t,k", [(1, 1), (1, 127), (3, 128), (5, 129), (70, 1000), (300, 1031), (64, 4096), (4097, 136)])
def test_quantize_rows(t, k, dtype):
    x = _normal((t, k), 1, dtype, 3.0)
    q, scale = mx.quantize_fp8(x)
    assert q.dtype == F8 and q.shape == (t, k) and scale.shape == (t, _blocks(k))
    _check_codes(x, q, scale)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("g,n,k", [(1, 1, 1), (2, 127, 129), (3, 128, 128), (1, 300, 1031), (4, 1000, 264)])
def test_quantize_weights(g, n, k, dtype):
    w = _normal((g, n, k), 1, dtype, 0.02)
    q, scale = mx.quantize_fp8_weight(w)
    _check_codes(w, q, scale)
    # the transposed weights have the transposed codes and scales
    qt, st = mx.quantize_fp8_weight(w.transpose(1, 2).contiguous())
    assert torch.equal(qt.view(torch.uint8), q.view(torch.uint8).transpose(1, 2))
    assert torch.equal(st, scale.transpose(1, 2))


@pytest.mark.parametrize("dtype", [BF, HF])
def test_every_value_under_many_scales(dtype):
    """Every finite value of the type beside largest ones of each size: borders between
    codes, subnormal codes, ties, scales down to the smallest numbers."""
    bits = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(dtype)
    finite = bits[torch.isfinite(bits)]
    size = finite.abs().float().sort(stable=True).indices
    values = finite[size]
    tops = [2 ** e * m for e in (-133, -130, -126, -120, -100, -20, -3, 0, 5, 15, 60, 120) for m in (1, 1.5, 1.109375, 1.75)]
    for top in tops:
        top = torch.tensor(top, dtype=torch.float64).to(dtype)
        if not 0 < float(top) < math.inf:
            continue
        fit = values[values.abs() <= top.to("cuda")]
        rows = min(len(fit) // 127, 300)
        if rows == 0:
            continue
        fit = fit[-127 * rows:]
        x = torch.cat([fit.view(-1, 127), top.to("cuda").expand(len(fit) // 127, 1)], 1).contiguous()
        _check_codes(x, *mx.quantize_fp8(x))


def test_ties_and_borders():
    """amax 448 * 2^e: the scale is a power of two and every border between codes is a value."""
    codes = torch.tensor(CODES, dtype=torch.float64)
    middle = (codes[1:] + codes[:-1]) / 2
    for e in (-120, -9, 0, 7):
        line = torch.cat([codes, middle, -middle]) * 2.0 ** e
        x = torch.full((3, 128), 448.0 * 2.0 ** e, dtype=torch.float64)
        x.view(-1)[:127], x.view(-1)[128:128 + 126], x.view(-1)[256:256 + 126] = line[:127], middle * 2.0 ** e, -middle * 2.0 ** e
        x = x.to(BF).cuda()
        q, scale = mx.quantize_fp8(x)
        assert (scale == 2.0 ** e).all()
        _check_codes(x, q, scale)


@pytest.mark.parametrize("exponent", [-80, 0, 40, 100, 110])
@pytest.mark.parametrize("k", [128, 131, 264])
def test_tiny_values_beside_borders(k, exponent):
    """A value on a border between two codes sends its neighbours of the same eight the exact way: those far
    below the scale are zeros of their sign, down to quotients that no number holds."""
    line = torch.zeros(k, dtype=torch.float64)
    tiny = [2.0 ** e for e in (-133, -126, -120, -110, -60, -30) if e < exponent - 12]
    for lane in range(0, min(k, 128) - 8, 8):
        line[lane] = 1.0625 * 2.0 ** exponent
        for i in range(7):
            line[lane + 1 + i] = (-1) ** (i + lane // 8) * tiny[(i + lane // 8) % len(tiny)]
    line[126], line[127] = -1.1875 * 2.0 ** exponent, 448.0 * 2.0 ** exponent
    x = torch.stack([line, -line, line.flip(0)]).to(BF).cuda()
    _check_codes(x, *mx.quantize_fp8(x))
    w = torch.stack([line, -line]).expand(3, 2, k).to(BF).contiguous().cuda()
    _check_codes(w, *mx.quantize_fp8_weight(w))


def test_special_rows():
    """Zeros, infinities and NaN: scale 0 or NaN with codes 0, the other blocks as they are."""
    x = _normal((6, 300), 1, BF)
    x[0] = 0
    x[1, :128] = -0.0
    x[2, 5], x[3, 200], x[4, 299] = math.inf, math.nan, -math.inf
    q, scale = mx.quantize_fp8(x)
    got = q.float()
    assert (scale[0] == 0).all() and (got[0] == 0).all() and scale[1, 0] == 0
    for r, b in ((2, 0), (3, 1), (4, 2)):
        assert torch.isnan(scale[r, b]) and (got[r, 128 * b:128 * b + 128] == 0).all()
        rest = [i for i in range(3) if i != b]
        assert torch.isfinite(scale[r, rest]).all()
    _check_codes(x[5:], q[5:], scale[5:])
    w = _normal((2, 130, 130), 2, BF)
    w[0, 129, 129] = math.nan
    q, scale = mx.quantize_fp8_weight(w)
    assert torch.isnan(scale[0, 1, 1]) and int(torch.isnan(scale).sum()) == 1
    assert (q[0, 128:, 128:].float() == 0).all()
    # the product is NaN where it meets the block, nowhere else
    xq, xs = mx.quantize_fp8(_normal((4, 130), 3, BF))
    y = mx.ragged_gemm_fp8(xq, xs, q, scale, _ms([2, 2]))
    assert torch.isnan(y[:2, 128:]).all() and not torch.isnan(y[:2, :128]).any() and not torch.isnan(y[2:]).any()


def test_strided_rows_and_buffers():
    wide = _normal((50, 400), 1, BF)
    for x in (wide[:, :300], wide[:, 3:140], wide[::2, 8:9]):
        q, scale = mx.quantize_fp8(x)
        _check_codes(x, q, scale)
        out = (torch.empty(x.shape, dtype=F8, device="cuda"),
               torch.empty((len(x), _blocks(x.shape[1])), device="cuda"))
        got = mx.quantize_fp8(x, out=out)
        assert got[0] is out[0] and torch.equal(out[0].view(torch.uint8), q.view(torch.uint8))
    q, scale = mx.quantize_fp8(wide[:0])
    assert q.shape == (0, 400) and scale.shape == (0, 4)


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------

def _spans(splits, rows):
    lo, got = 0, []
    for m in splits:
        got.append((min(lo, rows), min(lo + max(m, 0), rows)))
        lo += max(m, 0)
    return got


def _gather(x, index):
    if index is None:
        return x
    at = index.long()
    ok = (at >= 0) & (at < x.shape[0])
    return torch.where(ok[:, None], x[at.clamp(0, x.shape[0] - 1)], 0.0)


def _check(q, scale, w, w_scale, splits, index, got):
    """fp32 results: products of codes are exact, 128 of them are added in steps of at most 16,
    the scales' product, its product with the sum and the sum over blocks round once each.
    Results of 16 bits: the sum of a block may lose 2^-9 of its largest run of 8 products
    (16 partial sums, each cut 13 bits below the largest)."""
    x = q.double() * _spread(scale, q.shape)
    k = q.shape[1]
    for e, (lo, hi) in enumerate(_spans(splits, got.shape[0])):
        if hi == lo:
            continue
        a, b = _gather(x, index)[lo:hi], w[e].double() * _spread(w_scale, w.shape)[e]
        ref, mag = a @ b.T, a.abs() @ b.abs().T
        off = mag * (12 + 2 * _blocks(k)) * 2.0 ** -23
        if got.dtype != F32:
            for c in range(0, k, 128):
                top = torch.zeros_like(ref)
                for r in range(c, min(c + 128, k), 8):
                    r1 = min(r + 8, k)
                    top = torch.maximum(top, a[:, r:r1].abs() @ b[:, r:r1].abs().T)
                off += top * 2.0 ** -9
        fin = torch.finfo(got.dtype)
        tol = off + (ref.abs() + off) * fin.eps / 2 + fin.tiny * fin.eps
        assert not torch.isnan(got[lo:hi]).any(), e
        bad = (got[lo:hi].double() - ref).abs() > tol
        assert not bad.any(), (e, int(bad.sum()), float(((got[lo:hi].double() - ref).abs() / tol).max()))


def _case(tokens, splits, k, n, seed=1):
    q, scale = mx.quantize_fp8(_normal((tokens, k), seed, BF))
    w, w_scale = mx.quantize_fp8_weight(_normal((len(splits), n, k), seed + 1, BF, 0.02))
    return q, scale, w, w_scale


SPLITS = [
    [1],
    [0, 1, 0, 2, 0],
    [3, 0, 17, 1, 16, 15],
    [127, 128, 129, 0, 1],
    [255, 0, 256, 257, 63, 64, 65],
    [700, 5],
]
# (K, N): blocks that end inside the sizes, one or many, tiles of 16 bytes and not
WIDTHS = [(1, 1), (16, 16), (128, 128), (144, 264), (129, 130), (640, 520), (1000, 1031), (1031, 517), (1280, 256)]


@pytest.mark.parametrize("kn", WIDTHS)
@pytest.mark.parametrize("splits", SPLITS)
def test_products(splits, kn):
    k, n = kn
    case = _case(sum(splits), splits, k, n)
    for out in (BF, HF, F32):
        got = mx.ragged_gemm_fp8(*case, _ms(splits), out_dtype=out)
        _check(*case, splits, None, got)


@pytest.mark.parametrize("rows_each,g,k,n", [
    (1, 3, 4096, 1040), (16, 8, 2048, 1024), (20, 4, 1024, 264), (60, 2, 2048, 4096),   # few rows
    (31, 8, 2304, 8192), (90, 4, 4608, 4096), (300, 3, 1024, 4096),     # tiles of 64, 128 and 256 rows
    (2000, 2, 512, 5120), (700, 7, 896, 3000),                          # more tiles than a round
])
def test_forms(rows_each, g, k, n):
    splits = [rows_each + (i % 3) - 1 for i in range(g)]
    rows = sum(splits)
    case = _case(rows, splits, k, n)
    index = torch.randperm(rows, generator=torch.Generator().manual_seed(5)).int().cuda()
    for at in (None, index):
        for out in (BF, F32):
            _check(*case, splits, at, mx.ragged_gemm_fp8(*case, _ms(splits), row_index=at, out_dtype=out))


@pytest.mark.parametrize("kn", [(128, 256), (400, 264), (1031, 517)])
@pytest.mark.parametrize("tokens,splits", [(1, [1, 0, 1]), (40, [3, 0, 60, 17]), (300, [257, 0, 300, 343])])
def test_gather(tokens, splits, kn):
    """Any token any number of times; entries outside are rows of zeros of scale 0."""
    k, n = kn
    rows = sum(splits)
    index = torch.randint(0, tokens, (rows,), generator=torch.Generator().manual_seed(7)).int()
    if rows > 3:
        index[0], index[2], index[-1] = -1, tokens, 2 ** 31 - 1
    index = index.cuda()
    case = _case(tokens, splits, k, n)
    for out in (BF, F32):
        got = mx.ragged_gemm_fp8(*case, _ms(splits), row_index=index, out_dtype=out)
        _check(*case, splits, index, got)
        if rows > 3:
            # ... NaN where they meet a NaN of the weights or their scales
            w, ws = case[2].clone(), case[3].clone()
            w.view(torch.uint8)[0, 3, 5] = 0x7F
            ws[0, 0, 0] = math.inf if n > 200 else ws[0, 0, 0]
            bad = mx.ragged_gemm_fp8(case[0], case[1], w, ws, _ms(splits), row_index=index, out_dtype=out)
            assert torch.isnan(bad[0, 3]) and torch.isnan(bad[2, 3])
            assert torch.isnan(bad[0, :128]).all() and not torch.isnan(bad[0, 128:]).any()


@pytest.mark.parametrize("kn", [(128, 128), (400, 40), (1031, 517)])
@pytest.mark.parametrize("rows,splits", [(150, [5, 3]), (150, [5, -4, 3]), (150, [100, 200, 30]), (150, [0, 0, 0]),
                                         (700, [300, 5]), (700, [900, 1])])
def test_splits_that_do_not_fill_the_rows(rows, splits, kn):
    """Rows behind the last expert are neither read nor written; long splits are cut."""
    k, n = kn
    case = _case(rows, splits, k, n)
    end = max(hi for _, hi in _spans(splits, rows))
    case[0].view(torch.uint8)[end:] = 0x7F
    case[1][end:] = math.nan
    for dtype in (BF, F32):
        out = torch.full((rows, n), 7.0, dtype=dtype, device="cuda")
        assert mx.ragged_gemm_fp8(*case, _ms(splits), out_dtype=dtype, out=out) is out
        q, scale = case[0].clone(), case[1].clone()
        q.view(torch.uint8)[end:], scale[end:] = 0, 0
        _check(q, scale, *case[2:], splits, None, out)
        assert (out[end:] == 7.0).all()


@pytest.mark.parametrize("rows", [40, 600])
@pytest.mark.parametrize("k,n", [(384, 256), (208, 136)])
def test_strides_and_alignment(rows, k, n):
    splits = [rows - 7, 7]
    q, scale, w, w_scale = _case(rows, splits, k, n)
    for pad, shift in ((16, 0), (3, 0), (0, 1), (8, 8)):
        wide = torch.full((rows * (k + pad) + shift,), 0x7F, dtype=torch.uint8, device="cuda")
        qs = wide[shift:].view(rows, k + pad)[:, :k].view(F8)
        qs.view(torch.uint8).copy_(q.view(torch.uint8))
        buf = torch.full((rows * (n + pad) + shift,), 7.0, dtype=BF, device="cuda")
        out = buf[shift:].view(rows, n + pad)[:, :n]
        mx.ragged_gemm_fp8(qs, scale, w, w_scale, _ms(splits), out=out)
        _check(q, scale, w, w_scale, splits, None, out)
        assert (buf[:shift] == 7.0).all() and (buf[shift:].view(rows, n + pad)[:, n:] == 7.0).all()


@pytest.mark.parametrize("rows", [9, 300])
def test_exact_where_sums_are_small(rows):
    """Small whole numbers and scales that are powers of two: every form is exact."""
    gen = torch.Generator("cuda").manual_seed(3)
    k, n, splits = 640, 272, [rows - 2, 2]
    whole = lambda *s: torch.randint(-2, 3, s, generator=gen, device="cuda").float()  # noqa: E731
    power = lambda *s: 2.0 ** torch.randint(-2, 3, s, generator=gen, device="cuda").float()  # noqa: E731
    q, w = whole(rows, k).to(F8), whole(2, n, k).to(F8)
    scale, w_scale = power(rows, 5), power(2, 3, 5)
    x, ws = q.double() * _spread(scale, q.shape), w.double() * _spread(w_scale, w.shape)
    want = torch.cat([x[:rows - 2] @ ws[0].T, x[rows - 2:] @ ws[1].T])
    for out in (F32, BF, HF):
        got = mx.ragged_gemm_fp8(q, scale, w, w_scale, _ms(splits), out_dtype=out)
        assert torch.equal(got, want.to(out))


def test_captured_and_replayed():
    """Quantizer and product in one graph, replayed on new tokens with eager work between."""
    splits, k, n = [300, 0, 420, 100], 512, 768
    rows = sum(splits)
    ms = _ms(splits)
    x = _normal((rows, k), 1, BF)
    w, w_scale = mx.quantize_fp8_weight(_normal((4, n, k), 2, BF, 0.05))
    codes = (torch.empty((rows, k), dtype=F8, device="cuda"), torch.empty((rows, 4), device="cuda"))
    out = torch.empty((rows, n), dtype=BF, device="cuda")
    ws = torch.empty(max(1, mx.ragged_gemm_fp8_workspace_bytes(rows, rows, n, k, 4)), dtype=torch.uint8, device="cuda")

    def step():
        mx.quantize_fp8(x, out=codes)
        mx.ragged_gemm_fp8(*codes, w, w_scale, ms, out=out, workspace=ws)

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
        graph.replay()
        got = out.clone()
        want = mx.ragged_gemm_fp8(*mx.quantize_fp8(x), w, w_scale, ms)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


# few tiles of a long contraction: split among the CUs, each part four blocks and more, and joined.  Parts
# that begin inside a group of four blocks, a ragged last block, rows and columns past the tile's
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("splits,k,n", [
    ([200], 4096, 264), ([300], 4112, 4096), ([40, 300, 0, 260], 7184, 520), ([96, 95], 10128, 1032),
    ([32, 31, 33], 28688, 1032), ([257, 1300], 4112, 9000)])   # tiles of 128 and 64 rows; a round and a part of one
def test_few_tiles_of_long_sums(splits, k, n, dtype):
    rows = sum(splits)
    index = torch.randint(0, rows, (rows,), generator=torch.Generator().manual_seed(3), dtype=torch.int32).cuda()
    q, scale, w, w_scale = _case(rows, splits, k, n)
    for i in (None, index):
        got = mx.ragged_gemm_fp8(q, scale, w, w_scale, _ms(splits), row_index=i, out_dtype=dtype)
        _check(q, scale, w, w_scale, splits, i, got)
        assert torch.equal(got, mx.ragged_gemm_fp8(q, scale, w, w_scale, _ms(splits), row_index=i, out_dtype=dtype))


@pytest.mark.parametrize("splits,k,n", [([300, 0, 65, 128], 1031, 517), ([1300, 0, 1665, 1128], 257, 1801)])
def test_any_size_tiles(splits, k, n):
    """The any-size form with tiles of 64 and of 128 rows."""
    rows = sum(splits)
    index = torch.randint(-1, rows + 1, (rows,), generator=torch.Generator().manual_seed(4)).int().cuda()
    case = _case(rows, splits, k, n)
    for out in (F32, HF):
        _check(*case, splits, index, mx.ragged_gemm_fp8(*case, _ms(splits), row_index=index, out_dtype=out))
