"""Routing: choice, weights, row order, join, and their gradients, against
definitions written with numpy in float64."""

import math

import numpy as np
import pytest
import torch

import moe_expert_grouped_group_amd as mx

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]


def _route_ref(z, k, renorm, mask):
    """ids, weights, m_splits, row_token, row_pos by definition."""
    t, e = z.shape
    ids = np.full((t, k), -1, np.int32)
    w = np.zeros((t, k))
    prob = np.zeros((t, e))
    for i in range(t):
        ok = ~np.isnan(z[i]) & (z[i] > -np.inf) & mask[i]
        order = sorted((j for j in range(e) if ok[j]), key=lambda j: (-z[i, j], j))[:k]
        if not order:
            continue
        ids[i, :len(order)] = order
        over = order if renorm else [j for j in range(e) if ok[j]]
        ex = np.zeros(e)
        ex[over] = np.exp(z[i, over] - z[i, order[0]])
        prob[i] = ex / ex.sum()
        w[i, :len(order)] = prob[i, order]
    token, pos = np.full(t * k, -1, np.int32), np.full((t, k), -1, np.int32)
    splits, at = np.zeros(e, np.int64), 0
    for g in range(e):
        for i, j in zip(*np.nonzero(ids == g)):
            token[at], pos[i, j] = i, at
            at += 1
            splits[g] += 1
    return ids, w, splits, token, pos, prob


def _check_route(logits, k, renorm, mask=None, bwd=True):
    z = logits.double().cpu().numpy()
    m = np.ones(len(z), bool) if mask is None else mask.cpu().numpy().astype(bool)
    ids, w, splits, token, pos, prob = _route_ref(z, k, renorm, m)
    r = mx.moe_route(logits, k, renormalize=renorm, token_mask=mask)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    assert np.array_equal(r.m_splits.cpu().numpy(), splits)
    assert np.array_equal(r.row_token.cpu().numpy(), token)
    assert np.array_equal(r.row_pos.cpu().numpy(), pos)
    # exp of a difference (rounded to half a step of up to 2 |logit|), a sum of at
    # most E terms by halves, one division: a few fp32 steps, and those of the argument
    top = np.nanmax(np.where(np.isfinite(z), np.abs(z), 0), initial=1)
    tol = (8 + 2 * top + math.log2(z.shape[1]) + 16) * 2.0 ** -23
    assert np.all(np.abs(r.weights.cpu().numpy() - w) <= tol * w + 1e-37)
    if not bwd:
        return r
    d = torch.randn(w.shape, generator=torch.Generator().manual_seed(3))
    got = mx.moe_route_bwd(logits, r, d.cuda())
    full = np.zeros_like(prob)
    for i, j in zip(*np.nonzero(ids >= 0)):
        full[i, ids[i, j]] = d[i, j]
    inner = (prob * full).sum(1, keepdims=True)
    ref = prob * (full - inner)
    eps = torch.finfo(logits.dtype).eps / 2
    size = prob * (np.abs(full) + np.abs(prob * full).sum(1, keepdims=True))
    off = np.abs(got.double().cpu().numpy() - ref)
    assert np.all(off <= 3 * tol * size + eps * np.abs(ref) + torch.finfo(logits.dtype).smallest_normal)
    return r


def _logits(t, e, seed, dtype):
    gen = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn((t, e), generator=gen, device="cuda") * 2).to(dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (1, 8, 2), (5, 16, 16), (33, 17, 3), (64, 64, 8),
                                   (65, 100, 6), (256, 128, 8), (257, 256, 8), (300, 257, 4),
                                   (700, 512, 2), (1500, 1000, 10), (2000, 1024, 16), (129, 2, 1)])
def test_route(t, e, k, renorm, dtype):
    _check_route(_logits(t, e, t + e, dtype), k, renorm)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("t", [40, 900])
def test_route_ties_and_masks(t, renorm):
    """Equal logits go by lowest expert; -inf, the type's lowest value, NaN;
    tokens with fewer experts than top_k, with none, and masked ones."""
    gen = torch.Generator("cuda").manual_seed(1)
    z = torch.randint(-2, 3, (t, 24), generator=gen, device="cuda").float()
    z[1] = 0.0
    z[2] = -math.inf
    z[3] = -math.inf
    z[3, 20] = 1.0
    z[4] = torch.finfo(torch.float32).min
    z[5, ::2] = math.nan
    z[6] = math.nan
    z[7] = math.nan
    z[8, 3:] = torch.finfo(torch.float32).min
    mask = torch.rand(t, generator=gen, device="cuda") < 0.7
    mask[:9] = True
    mask[7] = False
    _check_route(z, 4, renorm)
    r = _check_route(z, 4, renorm, mask)
    assert (r.ids[2] == -1).all() and (r.ids[6] == -1).all() and r.ids[4].tolist() == [0, 1, 2, 3]
    assert torch.equal(r.ids, mx.moe_route(z, 4, renormalize=renorm, token_mask=mask.to(torch.uint8)).ids)
    none = torch.zeros_like(mask)
    r = _check_route(z, 4, renorm, none)
    assert (r.m_splits == 0).all() and (r.row_token == -1).all()


def test_route_all_tokens_to_the_same_experts():
    z = _logits(5000, 40, 1, torch.float32)
    z[:, 7] += 100
    z[:, 39] += 90
    r = _check_route(z, 2, True)
    assert r.m_splits[7] == 5000 and r.m_splits[39] == 5000


def test_route_no_tokens():
    r = mx.moe_route(torch.empty((0, 12), device="cuda"), 3)
    assert r.m_splits.tolist() == [0] * 12 and r.ids.shape == (0, 3)
    assert mx.moe_route_bwd(torch.empty((0, 12), device="cuda"), r, torch.empty((0, 3), device="cuda")).shape == (0, 12)


def test_route_large_against_sort():
    """More chunks than one launch of counts: order against a stable sort."""
    t, e, k = 200001, 64, 4
    z = _logits(t, e, 4, torch.bfloat16)
    r = mx.moe_route(z, k)
    value, order = torch.sort(z.float(), dim=1, descending=True, stable=True)
    assert torch.equal(r.ids, order[:, :k].int())
    flat = r.ids.flatten().long()
    rows = torch.argsort(flat, stable=True)
    assert torch.equal(r.row_token, (rows // k).int())
    pos = torch.empty_like(rows)
    pos[rows] = torch.arange(t * k, device="cuda")
    assert torch.equal(r.row_pos.flatten(), pos.int())
    assert torch.equal(r.m_splits, torch.bincount(flat, minlength=e))


def test_route_gradient_against_differences():
    z = torch.randn((6, 10), generator=torch.Generator().manual_seed(2)).double()
    d = torch.randn((6, 3), generator=torch.Generator().manual_seed(3)).double()
    for renorm in (True, False):
        r = mx.moe_route(z.float().cuda(), 3, renormalize=renorm)
        got = mx.moe_route_bwd(z.float().cuda(), r, d.float().cuda()).cpu().double()
        ids = r.ids.cpu().long()

        def loss(v):
            p = torch.softmax(v, 1).gather(1, ids)
            return float(((p / p.sum(1, keepdim=True) if renorm else p) * d).sum())

        h = 1e-5
        for i in range(6):
            for j in range(10):
                a, b = z.clone(), z.clone()
                a[i, j] += h
                b[i, j] -= h
                # second-order differences: h^2 times a third derivative of order 1, and
                # 1e-16 / h; the gradient itself is fp32
                assert abs((loss(a) - loss(b)) / (2 * h) - float(got[i, j])) < 1e-5


def _join_inputs(t, k, h, dtype, seed=0, missing=True):
    gen = torch.Generator("cuda").manual_seed(seed)
    rows = t * k
    y = torch.randn((rows, h), generator=gen, device="cuda").to(dtype)
    pos = torch.randperm(rows, generator=gen, device="cuda").view(t, k).int()
    if missing and rows > 4:
        pos.view(-1)[1] = -1
        pos.view(-1)[3] = rows
        pos[t // 2] = -1
    w = torch.rand((t, k), generator=gen, device="cuda")
    return y, pos, w, torch.randn((t, h), generator=gen, device="cuda").to(dtype)


@pytest.mark.parametrize("dtype", TYPES[1:])
@pytest.mark.parametrize("t,k,h", [(1, 1, 1), (1, 2, 7), (5, 8, 8), (33, 3, 1000), (9, 16, 520),
                                   (64, 6, 2049), (17, 4, 8199), (300, 2, 64)])
def test_join(t, k, h, dtype):
    y, pos, w, dout = _join_inputs(t, k, h, dtype)
    eps, f = torch.finfo(dtype).eps / 2, 2.0 ** -24
    tiny = torch.finfo(dtype).smallest_normal
    ok = (pos >= 0) & (pos < y.shape[0])
    rows = torch.where(ok[:, :, None], y.double()[pos.long().clamp(0, y.shape[0] - 1)], 0.0)
    for weights in (w, None):
        wd = (w if weights is not None else torch.ones_like(w)).double()
        ref = (rows * wd[:, :, None]).sum(1)
        mag = (rows.abs() * wd[:, :, None]).sum(1)
        got = mx.moe_combine(y, pos, weights)
        # a product and an addition of each of k terms, then the output's rounding
        assert ((got.double() - ref).abs() <= 2 * k * f * mag + eps * ref.abs() + tiny).all()
        dy = torch.full_like(y, 7.0)
        _, dw = mx.moe_combine_bwd(dout, y, pos, weights, out=(dy, None))
        refdy = torch.full_like(y, 7.0).double()
        refdy[pos[ok].long()] = (dout.double()[:, None, :] * wd[:, :, None])[ok]
        assert ((dy.double() - refdy).abs() <= (eps + 2 * f) * refdy.abs() + tiny).all()
        refdw = (rows * dout.double()[:, None, :]).sum(2)
        magdw = (rows * dout.double()[:, None, :]).abs().sum(2)
        # at most h / 256 / 8 * 8 + 10 additions in a row
        assert ((dw.double() - refdw).abs() <= (2 * h / 256 + 32) * f * magdw + 1e-37).all()
    only = mx.moe_combine_bwd(dout, y, pos, w, want_dy=False)
    assert only[0] is None and torch.equal(only[1], dw)
    only = mx.moe_combine_bwd(dout, y, pos, None, want_dweights=False)
    assert only[1] is None


def test_join_shifted_pointers():
    """Rows that start off 16 bytes."""
    y, pos, w, dout = _join_inputs(20, 4, 64, torch.bfloat16, missing=False)
    flat = torch.zeros(y.numel() + 3, dtype=torch.bfloat16, device="cuda")
    ys = flat[3:].view(y.shape)
    ys.copy_(y)
    assert torch.equal(mx.moe_combine(ys, pos, w), mx.moe_combine(y, pos, w))
    a, b = mx.moe_combine_bwd(dout, ys, pos, w), mx.moe_combine_bwd(dout, y, pos, w)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_join_infinities_stay_in_their_token():
    y, pos, w, _ = _join_inputs(50, 4, 40, torch.bfloat16, missing=False)
    clean = mx.moe_combine(y, pos, w)
    y[int(pos[7, 2])] = math.nan
    got = mx.moe_combine(y, pos, w)
    keep = torch.arange(50, device="cuda") != 7
    assert torch.equal(got[keep], clean[keep]) and torch.isnan(got[7]).all()


def test_routing_graph_replays():
    t, e, k, h = 600, 32, 4, 72
    z = _logits(t, e, 1, torch.float32)
    y = torch.randn((t * k, h), device="cuda").to(torch.bfloat16)
    dout = torch.randn((t, h), device="cuda").to(torch.bfloat16)
    ws = torch.empty(max(1, mx.moe_route_workspace_bytes(t, e)), dtype=torch.uint8, device="cuda")
    r = mx.moe_route(z, k, workspace=ws)
    out, dy, dz = torch.empty((t, h), dtype=y.dtype, device="cuda"), torch.empty_like(y), torch.empty_like(z)
    dw = torch.empty((t, k), device="cuda")

    def step():
        mx.moe_route(z, k, out=r, workspace=ws)
        mx.moe_combine(y, r.row_pos, r.weights, out=out)
        mx.moe_combine_bwd(dout, y, r.row_pos, r.weights, out=(dy, dw))
        mx.moe_route_bwd(z, r, dw, out=dz)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    held = (r.ids, r.weights, r.m_splits, r.row_token, r.row_pos, out, dy, dw, dz)
    for i in range(4):
        z.copy_(_logits(t, e, 20 + i, torch.float32))
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in held]
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, held):
            assert torch.equal(a, b)
