"""The rotary and norm kernels at layer sizes: several heads a unit, several
batches of them, several token tiles a block, a weight row for each head in
several planes.  (With few tokens every head is a unit of its own and every tile
a block: test_gpu_rope.)  Bounds as there; dweight: a thread adds at most two
tiles of twelve heads and a block its 32 groups in fp32, the rest is in 64 bits:
(24 + 32 + 8) E."""
import numpy as np
import pytest
import torch

import oracle
import block_sparse_attention_16_b200 as lbsa
from parity import host
from test_gpu_rope import E, HALF, _normal, _pair_size, _within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)
    lbsa.lbsa_device_status(clear=True)
    yield
    torch.cuda.synchronize()
    assert lbsa.lbsa_device_status() == 0


GRID, TAIL = (9, 29, 31), 13                # 8,104 tokens: 507 tiles of 16 (d = 128), 254 of 32 (d = 64)
N = 9 * 29 * 31 + TAIL


@pytest.mark.parametrize("weights", ["shared", "per_head"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,Hq,Hk,d,dims,layout", [(1, 12, 5, 128, (44, 42, 42), "interleaved"),
                                                   (2, 12, 5, 64, (16, 24, 24), "half"),
                                                   (1, 12, 5, 128, (32, 16, 16), "half"),
                                                   (2, 7, 3, 64, (20, 22, 22), "interleaved")])
def test_many_heads_and_tokens(B, Hq, Hk, d, dims, layout, dtype, weights):
    perm = torch.randperm(N, generator=torch.Generator().manual_seed(3)).to(torch.int32).cuda()
    take = perm.cpu().numpy()
    table, angles = lbsa.lbsa_rope_table(GRID, dims), oracle.rope_angles(GRID, dims, N)
    pos = dict(table=table, grid=GRID, dims=dims, perm=perm, layout=layout)
    xs = [_normal(i, B, N, H, d, dtype=dtype).transpose(1, 2) for i, H in enumerate((Hq, Hk, Hk))]
    ws = [1 + 0.3 * _normal(20 + i, *((H, d) if weights == "per_head" else (d,))) for i, H in enumerate((Hq, Hk))]
    ins, wts = xs, [*ws, None]
    ys = lbsa.lbsa_norm_rope(ins, wts, **pos)
    assert torch.equal(ys[2], xs[2][:, :, perm.long()])
    dys = [torch.empty_like(x).copy_(_normal(30 + i, *x.shape)) for i, x in enumerate(xs)]
    dxs, dws = lbsa.lbsa_norm_rope_backward(dys, ins, wts, **pos)
    again = lbsa.lbsa_norm_rope_backward(dys, ins, wts, **pos)
    assert dws[2] is None
    moved = torch.empty_like(dys[2])
    moved[:, :, perm.long()] = dys[2]
    assert torch.equal(dxs[2], moved)
    turned = lbsa.lbsa_rope(xs, **pos)
    back = lbsa.lbsa_rope(dys, inverse=True, **pos)
    for i, x in enumerate(xs):
        x64, dy = host(x).astype(np.float64), np.empty(x.shape)
        dy[:, :, take] = host(dys[i])
        for got, src, inverse in ((turned[i], x64, False), (back[i], dy, True)):
            ref = oracle.rope_rotate(src, angles, layout, inverse=inverse)
            bound = HALF[dtype] * np.abs(ref) + 6 * E * _pair_size(src, angles, layout)
            _within(host(got), ref if inverse else ref[:, :, take], bound if inverse else bound[:, :, take])
        if i == 2:
            continue
        w64 = host(ws[i]).astype(np.float64)
        ref = oracle.norm_rope(x64, w64, angles, layout)
        bound = HALF[dtype] * np.abs(ref) + 24 * E * _pair_size(oracle.norm_rope(x64, w64), angles, layout)
        _within(host(ys[i]), ref[:, :, take], bound[:, :, take])
        rdx, rdw = oracle.norm_rope_grad(dy, x64, w64, angles, layout)
        r = 1 / np.sqrt((x64 * x64).mean(-1, keepdims=True) + 1e-6)
        n, wr = x64 * r, (w64 if w64.ndim == 1 else w64[:, None])
        size = _pair_size(dy, angles, layout)
        slack = 32 * E * r * (size * np.abs(wr) + np.abs(n) * (size * np.abs(wr * n)).mean(-1, keepdims=True))
        _within(host(dxs[i]), rdx, HALF[dtype] * np.abs(rdx) + slack)
        total = (size * np.abs(n)).sum((0, 2))
        total = total.sum(0) if w64.ndim == 1 else total
        assert dws[i].dtype == torch.float32 and dws[i].shape == ws[i].shape
        _within(host(dws[i]), rdw, 64 * E * total)
        assert torch.equal(dws[i], again[1][i]) and torch.equal(dxs[i], again[0][i])


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_gradients_without_an_eps(dtype, per_head):
    # five heads in batches of two or four and a ragged last tile: rows that are not there have 1 / sqrt(0)
    n, d = 2407, 128
    x, dy = _normal(1, 1, 5, n, d, dtype=dtype), _normal(2, 1, 5, n, d, dtype=dtype)
    w = 1 + 0.2 * _normal(3, *((5, d) if per_head else (d,)))
    y, = lbsa.lbsa_norm_rope([x], [w], eps=0.0)
    (dx,), (dw,) = lbsa.lbsa_norm_rope_backward([dy], [x], [w], eps=0.0)
    x64, dy64, w64 = (host(t).astype(np.float64) for t in (x, dy, w))
    ref = oracle.norm_rope(x64, w64, eps=0.0)
    _within(host(y), ref, (HALF[dtype] + 24 * E) * np.abs(ref))
    rdx, rdw = oracle.norm_rope_grad(dy64, x64, w64, eps=0.0)
    r = 1 / np.sqrt((x64 * x64).mean(-1, keepdims=True))
    nrm, wr = x64 * r, (w64[:, None] if per_head else w64)
    slack = 32 * E * r * (np.abs(dy64 * wr) + np.abs(nrm) * np.abs(dy64 * wr * nrm).mean(-1, keepdims=True))
    _within(host(dx), rdx, HALF[dtype] * np.abs(rdx) + slack)
    _within(host(dw), rdw, 64 * E * np.abs(dy64 * nrm).sum((0, 2) if per_head else (0, 1, 2)))
