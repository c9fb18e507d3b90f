"""Rotary positions, the per-head norm with rotation, and its gradients on the
GPU against the fp64 oracle.

Bounds (E = 2^-24, one fp32 rounding; h = half a step of the output's type,
2^-8 for bf16, 2^-24 for fp32):
  rotation   |err| <= h |ref| + 6 E (|a| + |b|): table entry, two products, one
             sum, each off by E relative to their own size
  norm       the sum of squares (8 per lane, 4 shuffles), its mean, eps, the
             reciprocal root (2 ulp = 4 E) and two products: below 24 E in all
  gradient   dx = r (dn - n mean(dn n)): 32 E of r (|dn pair| + |n| mean |dn n|)
  dweight    per column sums of M products in fp32 of at most L in a row and
             then at most 32: (L + 64) E sum |du n|
"""
import numpy as np
import pytest
import torch

import oracle
import block_sparse_attention_16_b200 as lbsa
from parity import host

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: E}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)
    lbsa.lbsa_device_status(clear=True)
    yield
    torch.cuda.synchronize()
    assert lbsa.lbsa_device_status() == 0


def _normal(seed, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


def _pair_size(x, angles, layout):
    """|a| + |b| of every element's pair (the element itself where it has none)."""
    x, rd = np.abs(x), 2 * angles.shape[1]
    out = x.copy()
    i = np.arange(rd // 2)
    a, b = (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + rd // 2)
    out[..., a] = out[..., b] = x[..., a] + x[..., b]
    return out


def _within(got, ref, bound):
    bad = ~(np.abs(got - ref) <= bound)                      # a NaN is off, too
    assert not bad.any(), f"{bad.sum()} of {bad.size} off; worst {np.max(np.abs(got - ref) / np.maximum(bound, 1e-300)):.3g}x of its bound"


CASES = [
    # B, Hq, Hk, d, grid, dims, layout, dtype, perm, tail, start
    (1, 1, 1, 64, (1, 1, 1), (22, 20, 22), "interleaved", torch.bfloat16, None, 0, (9001, 0, 0)),     # one token
    (1, 12, 12, 128, (1, 1, 1), (44, 42, 42), "interleaved", torch.float32, None, 0, (7, 1, 2)),
    (2, 3, 1, 128, (3, 7, 11), (44, 42, 42), "interleaved", torch.bfloat16, "3d", 0, (0, 0, 0)),
    (1, 6, 2, 64, (2, 5, 9), (16, 24, 24), "half", torch.bfloat16, "random", 13, (100, 0, 0)),
    (2, 5, 5, 64, (3, 7, 9), (2, 0, 4), "interleaved", torch.float32, "3d", 1, (0, 0, 0)),            # part of the row
    (1, 4, 2, 128, (1, 15, 13), (0, 64, 64), "half", torch.float32, None, 0, (0, 3, 5)),              # two axes
    (1, 2, 2, 128, (40, 1, 1), (96, 0, 0), "half", torch.bfloat16, "random", 0, (50000, 0, 0)),       # one axis, far away
]


def _inputs(case, strided):
    B, Hq, Hk, d, grid, dims, layout, dtype, order, tail, start = case
    n = grid[0] * grid[1] * grid[2] + tail
    xs = [_normal(i, B, n, H, d, dtype=dtype).transpose(1, 2) for i, H in enumerate((Hq, Hk))]
    if not strided:
        xs = [x.contiguous() for x in xs]
    perm = None
    if order == "random":
        perm = torch.randperm(n, generator=torch.Generator().manual_seed(3)).to(torch.int32).cuda()
    elif order == "3d":
        perm = torch.cat([lbsa.lbsa_partition_perm(*grid, "3d"), torch.arange(n - tail, n, dtype=torch.int32)]).cuda()
    table = lbsa.lbsa_rope_table(grid, dims, start=start)
    angles = oracle.rope_angles(grid, dims, n, start=start)
    take = np.arange(n) if perm is None else perm.cpu().numpy()
    return xs, perm, table, angles, take


def test_table_is_the_rounded_angle():
    grid, dims = (5, 3, 7), (44, 42, 42)
    t = lbsa.lbsa_rope_table(grid, dims, theta=500.0, start=(123456, 0.5, -3)).cpu().double().numpy()
    rows = []
    for extent, m, first in zip(grid, dims, (123456, 0.5, -3)):
        rows.append(((first + np.arange(extent))[:, None] * 500.0 ** (-2.0 * np.arange(m // 2) / m)).reshape(-1))
    ang = np.concatenate(rows)
    # an angle of 1.2e5 in 64 bits is off by 1.2e5 * 2^-52 or so, far below a rounding to fp32
    assert np.abs(t[:, 0] - np.cos(ang)).max() <= E and np.abs(t[:, 1] - np.sin(ang)).max() <= E


@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
def test_rope_and_its_inverse(case, strided):
    grid, dims, layout, dtype = case[4:8]
    xs, perm, table, angles, take = _inputs(case, strided)
    ys = lbsa.lbsa_rope(xs, table, grid, dims, perm, layout=layout)
    for x, y in zip(xs, ys):
        assert y.stride() == torch.empty_like(x).stride()
        ref = oracle.rope_rotate(host(x), angles, layout)
        bound = HALF[dtype] * np.abs(ref) + 6 * E * _pair_size(host(x).astype(np.float64), angles, layout)
        _within(host(y), ref[:, :, take], bound[:, :, take])
    # the inverse (= the gradient for dy = ys) comes back into source order
    back = lbsa.lbsa_rope(ys, table, grid, dims, perm, inverse=True, layout=layout)
    for y, b in zip(ys, back):
        src = np.empty_like(host(y), dtype=np.float64)
        src[:, :, take] = host(y)
        ref = oracle.rope_rotate(src, angles, layout, inverse=True)
        _within(host(b), ref, HALF[dtype] * np.abs(ref) + 6 * E * _pair_size(src, angles, layout))


@pytest.mark.parametrize("weights", ["shared", "per_head", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
def test_norm_rope_and_gradients(case, weights):
    grid, dims, layout, dtype = case[4:8]
    xs, perm, table, angles, take = _inputs(case, strided=weights == "shared")
    v = _normal(8, *xs[1].shape, dtype=dtype)
    d = xs[0].shape[-1]
    ws = [1 + 0.3 * _normal(20 + i, *((x.shape[1], d) if weights == "per_head" else (d,))) for i, x in enumerate(xs)]
    ws = [w.bfloat16() for w in ws] if weights == "bf16" else ws
    ins, wts = [*xs, v], [*ws, None]
    ys = lbsa.lbsa_norm_rope(ins, wts, table, grid, dims, perm, layout=layout)
    assert torch.equal(ys[2], v if perm is None else v[:, :, perm.long()])
    dys = [torch.empty_like(x).copy_(_normal(30 + i, *x.shape)) for i, x in enumerate(ins)]
    dxs, dws = lbsa.lbsa_norm_rope_backward(dys, ins, wts, table, grid, dims, perm, layout=layout)
    again = lbsa.lbsa_norm_rope_backward(dys, ins, wts, table, grid, dims, perm, layout=layout)
    assert dws[2] is None
    if perm is not None:
        moved = torch.empty_like(dys[2])
        moved[:, :, perm.long()] = dys[2]
        assert torch.equal(dxs[2], moved)
    for i, (x, w) in enumerate(zip(xs, ws)):
        x64, w64 = host(x).astype(np.float64), host(w).astype(np.float64)
        u = oracle.norm_rope(x64, w64)
        ref = oracle.norm_rope(x64, w64, angles, layout)
        bound = HALF[dtype] * np.abs(ref) + 24 * E * _pair_size(u, angles, layout)
        _within(host(ys[i]), ref[:, :, take], bound[:, :, take])
        dy = np.empty(dys[i].shape)
        dy[:, :, take] = host(dys[i])
        rdx, rdw = oracle.norm_rope_grad(dy, x64, w64, angles, layout)
        r = 1 / np.sqrt((x64 * x64).mean(-1, keepdims=True) + 1e-6)
        n, wr = x64 * r, (w64 if w64.ndim == 1 else w64[:, None])
        size = _pair_size(dy, angles, layout)
        slack = 32 * E * r * (size * np.abs(wr) + np.abs(n) * (size * np.abs(wr * n)).mean(-1, keepdims=True))
        _within(host(dxs[i]), rdx, HALF[dtype] * np.abs(rdx) + slack)
        total = (size * np.abs(n)).sum((0, 2))
        total = total.sum(0) if w64.ndim == 1 else total
        longest = 4 * (-(-x.shape[2] // 16))
        assert dws[i].dtype == torch.float32 and dws[i].shape == w.shape
        _within(host(dws[i]), rdw, (longest + 64) * E * total)
        assert torch.equal(dws[i], again[1][i]) and torch.equal(dxs[i], again[0][i])


def test_norm_without_rotation_and_zero_rows():
    x, w = _normal(1, 1, 2, 33, 64), 1 + 0.2 * _normal(2, 64)
    x[:, :, 4] = 0                                            # 1 / sqrt(eps), not infinity
    y, = lbsa.lbsa_norm_rope([x], [w])
    ref = oracle.norm_rope(host(x), host(w))
    _within(host(y), ref, E * np.abs(ref) + 24 * E * np.abs(ref))
    (dx,), (dw,) = lbsa.lbsa_norm_rope_backward([torch.ones_like(x)], [x], [w])
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()
    assert not y[:, :, 4].any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout,dims", [("interleaved", (6, 0, 4)), ("half", (16, 0, 16))])
def test_what_keeps_its_place_is_copied(layout, dims, dtype):
    # text tokens past the grid and elements past the rotated ones: infinities, NaN and -0 too
    x = _normal(1, 1, 3, 29, 64, dtype=dtype)
    rd = sum(dims)
    odd = torch.tensor([float("inf"), 1.0, float("-inf"), float("nan"), -0.0, 2.0], device="cuda", dtype=dtype)
    x[..., 24:, :] = odd.repeat(11)[:64]
    x[..., rd:] = odd.repeat(10)[:64 - rd]
    table = lbsa.lbsa_rope_table((2, 3, 4), dims)
    for inverse in (False, True):
        y, = lbsa.lbsa_rope([x], table, (2, 3, 4), dims, layout=layout, inverse=inverse)
        assert torch.isfinite(y[..., :24, :rd]).all() and not torch.equal(y[..., :24, :rd], x[..., :24, :rd])
        for got, want in ((y[..., 24:, :], x[..., 24:, :]), (y[..., rd:], x[..., rd:])):
            assert torch.equal(got.isnan(), want.isnan())
            assert torch.equal(got.nan_to_num(9.0, posinf=99.0, neginf=-99.0), want.nan_to_num(9.0, posinf=99.0, neginf=-99.0))
            assert torch.equal(got.signbit() & ~want.isnan(), want.signbit() & ~want.isnan())


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradients_without_an_eps(dtype, per_head):
    # odd heads and tokens: the last tile's and batch's rows that are not there have 1 / sqrt(0)
    x, dy = _normal(1, 1, 3, 37, 128, dtype=dtype), _normal(2, 1, 3, 37, 128, dtype=dtype)
    w = 1 + 0.2 * _normal(3, *((3, 128) if per_head else (128,)))
    (dx,), (dw,) = lbsa.lbsa_norm_rope_backward([dy], [x], [w], eps=0.0)
    x64, dy64, w64 = (host(t).astype(np.float64) for t in (x, dy, w))
    rdx, rdw = oracle.norm_rope_grad(dy64, x64, w64, eps=0.0)
    r = 1 / np.sqrt((x64 * x64).mean(-1, keepdims=True))
    n, wr = x64 * r, (w64[:, None] if per_head else w64)
    slack = 32 * E * r * (np.abs(dy64 * wr) + np.abs(n) * np.abs(dy64 * wr * n).mean(-1, keepdims=True))
    _within(host(dx), rdx, HALF[dtype] * np.abs(rdx) + slack)
    total = np.abs(dy64 * n).sum((0, 2) if per_head else (0, 1, 2))
    _within(host(dw), rdw, (3 * 3 + 64) * E * total)          # at most three token tiles, three heads in a row


def test_bad_perm_entries_skip_their_row_and_are_reported():
    x, table = _normal(1, 1, 2, 24, 64), lbsa.lbsa_rope_table((2, 3, 4), (16, 24, 24))
    perm = torch.arange(24, dtype=torch.int32, device="cuda")
    whole, = lbsa.lbsa_rope([x], table, (2, 3, 4), (16, 24, 24))
    perm[5], perm[9] = 24, -1
    y = torch.full_like(x, 7.0)
    lbsa.lbsa_rope([x], table, (2, 3, 4), (16, 24, 24), perm, outs=[y])
    assert lbsa.lbsa_device_status(clear=True) == lbsa.LBSA_ERR_BAD_INDEX
    good = [i for i in range(24) if i not in (5, 9)]
    assert torch.equal(y[:, :, good], whole[:, :, good]) and (y[:, :, [5, 9]] == 7).all()
    dx = torch.full_like(x, 7.0)
    lbsa.lbsa_norm_rope_backward([x], [x], [torch.ones(64, device="cuda")], table, (2, 3, 4), (16, 24, 24), perm, dxs=[dx])
    assert lbsa.lbsa_device_status(clear=True) == lbsa.LBSA_ERR_BAD_INDEX
    assert (dx[:, :, [5, 9]] == 7).all() and (dx[:, :, good] != 7).any()


def test_rows_between_tensors_stay_as_they_are():
    # heads of a wider buffer: nothing outside the output's own rows is written
    x, w = _normal(1, 1, 3, 37, 64), torch.ones(64, device="cuda")
    buf = torch.full((1, 37, 5, 64), 3.0, device="cuda")
    y = buf.transpose(1, 2)[:, 1:4]
    lbsa.lbsa_norm_rope([x], [w], outs=[y])
    plain, = lbsa.lbsa_norm_rope([x], [w])
    assert torch.equal(y, plain) and (buf[:, :, [0, 4]] == 3).all()


def test_streams_and_captured_graphs():
    grid, dims = (3, 7, 11), (44, 42, 42)
    x, w, table = _normal(1, 1, 4, 231, 128, dtype=torch.bfloat16), 1 + 0.1 * _normal(2, 128), lbsa.lbsa_rope_table(grid, dims)
    dy = _normal(3, 1, 4, 231, 128, dtype=torch.bfloat16)
    perm = lbsa.lbsa_partition_perm(*grid, "3d", device="cuda")

    def step():
        y, = lbsa.lbsa_norm_rope([x], [w], table, grid, dims, perm)
        (dx,), (dw,) = lbsa.lbsa_norm_rope_backward([dy], [x], [w], table, grid, dims, perm)
        return y, dx, dw
    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        other = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, step()))
    x.mul_(-1)
    for g, _ in graphs:                                        # back to back, each with its own scratch
        g.replay()
    torch.cuda.synchronize()
    want = step()
    for _, got in graphs:
        assert all(torch.equal(a, b) for a, b in zip(want, got))
