"""Gradients of block-sparse attention on the GPU against the fp64 oracle.

Bounds, element by element (E = 2^-24; h = half a step of the type, 2^-8 for
bf16, E for fp32; |.| sums over the kept pairs):
  P      relative p = 4 E (|s| + |lse| + 4) + d E scale (|q|.|k|): the logit's sum
         of d products, its scaling, lse and the exponential's argument; for bf16
         + 2^-13 (a cubic exponential, 8e-5) + h (P rounded for the products)
  out    (p + h) sum P |v| + h |out|, from the forward call
  D      sum |dout| (error of out) + d E sum |dout| |out|
  dS     (p + h') |dS| + P (error of D + d E sum |dout| |v|), h' = h for bf16
  dv     sum (p + h') P |dout| + n E sum P |dout| + h |dv|
  dq     scale (sum (error of dS) |k| + n E sum |dS| |k|) + h |dq|; dk alike
"""
import numpy as np
import pytest
import torch

import oracle
import block_sparse_attention_16_b200 as lbsa
from parity import gpu_csr, host

pytestmark = pytest.mark.gpu
E = 2.0 ** -24


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


def _pairs(keep, N, block, per_token):
    """Kept (query, key) pairs [B, H, N, N] of block (or token) lists."""
    p = np.repeat(keep, block, 3)[..., :N]
    return p if per_token else np.repeat(p, block, 2)[:, :, :N]


def _blockset(keep, block, per_token=False):
    """A blockset that keeps exactly `keep` [B, H, rows, nB]."""
    if per_token:
        # equal weights: all of them are needed to reach this share
        return lbsa.lbsa_select_tokens(torch.from_numpy(keep).cuda().float() * 0.5, block, 1 - 2.0 ** -24)
    B, H, nB, _ = keep.shape
    rp, col = oracle.csr_from_rows([np.nonzero(r)[0] for r in keep.reshape(-1, nB)])
    return lbsa.lbsa_blockset_from_csr(torch.from_numpy(rp).cuda(), torch.from_numpy(col).cuda(), B, H, nB, block)


def _reference(q, k, v, dout, pairs, dtype):
    """((dq, dk, dv), their bounds) in fp64, dense."""
    q, k, v, dout = (host(x).astype(np.float64) for x in (q, k, v, dout))
    N, d = q.shape[2:]
    scale, t = d ** -0.5, lambda x: x.swapaxes(-1, -2)      # noqa: E731
    h = 2.0 ** -8 if dtype == torch.bfloat16 else E
    hp = h if dtype == torch.bfloat16 else 0.0
    s = (q @ t(k)) * scale
    z = np.where(pairs, s, -np.inf)
    m = np.where(pairs.any(-1, keepdims=True), z.max(-1, keepdims=True), 0.0)
    e = np.exp(z - m)
    l = e.sum(-1, keepdims=True)
    p = e / np.where(l > 0, l, 1.0)
    lse = np.where(l > 0, m + np.log(np.where(l > 0, l, 1.0)), 0.0)
    out, dp = p @ v, dout @ t(v)
    ds = p * (dp - (p * dp).sum(-1, keepdims=True))
    grads = scale * (ds @ k), scale * (t(ds) @ q), t(p) @ dout
    a = np.abs
    pe = 4 * E * (a(s) + a(lse) + 4) + d * E * scale * (a(q) @ t(a(k)))
    if dtype == torch.bfloat16:
        pe = pe + 2.0 ** -13
    oe = (p * (pe + hp)) @ a(v) + (h + N * E) * a(out)
    de = (a(dout) * oe).sum(-1, keepdims=True) + d * E * (a(dout) * a(out)).sum(-1, keepdims=True)
    dse = (pe + hp) * a(ds) + p * (de + d * E * (a(dout) @ t(a(v))))
    n = N * E
    # bf16: dq is summed as sum_c dS_rc (k_c - m), the same number for any m since sum_c dS_rc = 0, with m the mean
    # of the 64-row piece nearest to the row's own that its 128-row tile keeps (of two the later): an error of dS_rc
    # counts |k_c - m|, the fp32 sums are of |dS_rc| |k_c| and |dS_rc| |m|
    dq_bound = np.empty_like(q)
    for t0 in range(0, N, 64):
        rows, m = slice(t0, t0 + 64), 0.0
        if dtype == torch.bfloat16:
            tile = slice(t0 // 128 * 128, t0 // 128 * 128 + 128)
            on = np.add.reduceat(pairs[:, :, tile].any(2), np.arange(0, N, 64), axis=-1) > 0
            away = np.abs(np.arange(on.shape[-1]) - t0 // 64) * 2 + (np.arange(on.shape[-1]) < t0 // 64)
            near = np.where(on, away, 1 << 30)
            on = on & (near == near.min(-1, keepdims=True))
            on = np.repeat(on, 64, -1)[..., :N, None]
            m = ((on * k).sum(2) / np.maximum(on.sum(2), 1))[:, :, None]
        dq_bound[:, :, rows] = scale * (dse[:, :, rows] @ a(k - m) + n * a(ds[:, :, rows]) @ (a(k) + a(m)))
    bounds = (dq_bound + h * a(grads[0]), scale * (t(dse + n * a(ds)) @ a(q)) + h * a(grads[1]),
              t(p * (pe + hp + n)) @ a(dout) + h * a(grads[2]))
    return grads, bounds


def _check(got, ref, bounds, names=("dq", "dk", "dv")):
    for name, g, r, b in zip(names, got, ref, bounds):
        g = host(g).astype(np.float64)
        assert np.isfinite(g).all(), f"{name}: not finite"
        bad = np.abs(g - r) > b + 1e-30
        assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size} off, worst "
                               f"{np.max(np.abs(g - r) / (b + 1e-30)):.3g}x of its bound at {np.argwhere(bad)[0]}")


def _run(B, H, N, d, block, dtype, keep, per_token=False, seed=0, sharp=1.0, view=None):
    q, k, v, dout = (_normal(seed + i, B, H, N, d, dtype=dtype) * (sharp if i == 0 else 1.0) for i in range(4))
    if view:
        q, k, v, dout = (view(x) for x in (q, k, v, dout))
    bs = _blockset(keep, block, per_token)
    out, lse = lbsa.lbsa_attend(q, k, v, bs, want_lse=True)
    got = lbsa.lbsa_attend_backward(q, k, v, bs, out, lse, dout)
    again = lbsa.lbsa_attend_backward(q, k, v, bs, out, lse, dout)
    assert lbsa.lbsa_get_status(bs) == 0
    for a, b in zip(got, again):
        assert torch.equal(a, b) and a.stride() == q.stride()
    ref, bounds = _reference(q, k, v, dout, _pairs(keep, N, block, per_token), dtype)
    _check(got, ref, bounds)
    return got


def _keep(seed, B, H, rows, nB, share):
    keep = np.random.default_rng(seed).random((B, H, rows, nB)) < share
    if rows > 1:
        keep[0, 0, rows // 2] = False                     # rows that keep nothing
        keep[-1, -1, rows - 1] = False
    if nB > 2:
        keep[0, 0, :, 1] = False                          # a key block that nobody keeps
    keep[:, :, 0, 0] = True
    return keep


BOTH = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])


@BOTH
@pytest.mark.parametrize("share", [0.15, 0.6, 1.0])
@pytest.mark.parametrize("B,H,N,d,block", [
    (1, 1, 1, 64, 64), (1, 2, 1, 128, 128), (1, 1, 63, 128, 64), (1, 2, 64, 64, 64), (2, 1, 65, 128, 64),
    (1, 1, 127, 64, 128), (1, 2, 128, 128, 128), (1, 2, 129, 64, 128), (2, 2, 288, 128, 64), (1, 3, 360, 128, 128),
    (1, 2, 210, 64, 64), (1, 2, 1024, 128, 64), (2, 1, 651, 64, 128), (1, 1, 1217, 128, 64), (1, 1, 833, 64, 64),
])
def test_block_lists(B, H, N, d, block, share, dtype):
    nB = -(-N // block)
    _run(B, H, N, d, block, dtype, _keep(N, B, H, nB, nB, share), seed=N + d)


@BOTH
@pytest.mark.parametrize("share", [0.1, 0.7])
@pytest.mark.parametrize("B,H,N,d", [(1, 1, 1, 128), (1, 2, 64, 64), (2, 1, 131, 128), (1, 2, 450, 64), (1, 1, 700, 128)])
def test_token_lists(B, H, N, d, share, dtype):
    _run(B, H, N, d, 64, dtype, _keep(N, B, H, N, -(-N // 64), share), per_token=True, seed=N + d)


@BOTH
def test_sharp_and_flat_rows(dtype):
    keep = _keep(5, 1, 2, 5, 5, 0.7)
    _run(1, 2, 290, 128, 64, dtype, keep, seed=5, sharp=12.0)     # logits to about 40: one key takes nearly all
    _run(1, 2, 290, 128, 64, dtype, keep, seed=5, sharp=0.0)      # equal logits


@BOTH
@pytest.mark.parametrize("d", [64, 128])
def test_keys_with_much_in_common(d, dtype):
    # sum_c dS_rc = 0 takes the common part out of dq; roundings of dS must not bring it back
    B, H, N, keep = 1, 2, 400, _keep(4, 1, 2, 7, 7, 0.6)
    q, k, v, dout = (_normal(4 + i, B, H, N, d, dtype=dtype) for i in range(4))
    k = (k + 20 * _normal(3, d)).to(dtype)
    bs = _blockset(keep, 64)
    out, lse = lbsa.lbsa_attend(q, k, v, bs, want_lse=True)
    got = lbsa.lbsa_attend_backward(q, k, v, bs, out, lse, dout)
    _check(got, *_reference(q, k, v, dout, _pairs(keep, N, 64, False), dtype))


@BOTH
def test_projection_strides(dtype):
    # [B, N, H, d] as a projection leaves it, seen as [B, H, N, d]
    keep = _keep(6, 2, 3, 4, 4, 0.5)
    _run(2, 3, 250, 64, 64, dtype, keep, seed=6, view=lambda x: x.transpose(1, 2).contiguous().transpose(1, 2))


@BOTH
def test_every_tensor_with_strides_of_its_own(dtype):
    B, H, N, d, keep = 2, 3, 200, 64, _keep(8, 2, 3, 4, 4, 0.6)
    q, k, v, dout = (_normal(60 + i, B, H, N, d, dtype=dtype) for i in range(4))
    bs = _blockset(keep, 64)
    out, lse = lbsa.lbsa_attend(q, k, v, bs, want_lse=True)
    want = lbsa.lbsa_attend_backward(q, k, v, bs, out, lse, dout)

    def other(x, i):                                      # rows apart, heads innermost, batches in a wider buffer
        if i % 3 == 0:
            return x.transpose(1, 2).contiguous().transpose(1, 2)
        buf = torch.full((B, H + 1, N + i, d + 8 * i), float("nan"), dtype=x.dtype, device=x.device)
        buf[:, :H, :N, :d] = x
        return buf[:, :H, :N, :d]
    ins = [other(x, i) for i, x in enumerate((q, k, v, out, dout))]
    outs = [other(torch.zeros_like(q), i) for i in (4, 3, 2)]
    lbsa.lbsa_attend_backward(*ins[:3], bs, ins[3], lse, ins[4], *outs)
    for a, b in zip(outs, want):
        assert torch.equal(a, b)
    for a, b in zip(lbsa.lbsa_attend_backward(*ins[:3], bs, ins[3], lse, ins[4]), want):
        assert torch.equal(a, b)


@BOTH
def test_rows_past_the_last_token_are_neither_read_nor_written(dtype):
    N, keep = 150, _keep(7, 1, 2, 3, 3, 0.7)
    bufs = [_normal(70 + i, 1, 2, 192, 64, dtype=dtype) for i in range(4)]
    q, k, v, dout = (x[:, :, :N] for x in bufs)
    bs = _blockset(keep, 64)
    outs = [torch.full_like(bufs[0], 5.0) for _ in range(4)]
    out, lse = lbsa.lbsa_attend(q, k, v, bs, out=outs[0][:, :, :N], want_lse=True)
    want = [g.clone() for g in lbsa.lbsa_attend_backward(q, k, v, bs, out, lse, dout, *(o[:, :, :N] for o in outs[1:]))]
    for o in outs:
        assert (o[:, :, N:] == 5.0).all()
    for x in bufs + outs[:1]:
        x[:, :, N:] = float("nan")
    got = lbsa.lbsa_attend_backward(q, k, v, bs, out, lse, dout, *(o[:, :, :N] for o in outs[1:]))
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    ref, bounds = _reference(q, k, v, dout, _pairs(keep, N, 64, False), dtype)
    _check(got, ref, bounds)


@BOTH
@pytest.mark.parametrize("scope", ["row", "head", "routed", "local_topk"])
def test_selected_blocksets(scope, dtype):
    # the whole path: scores, a selection, attention and its gradients
    q, k, v, dout = (_normal(80 + i, 1, 3, 500, 64, dtype=dtype) for i in range(4))
    scores = lbsa.lbsa_score(q, k, 64)
    bs = (lbsa.lbsa_select(scores, 64, 0.6, "row") if scope == "row" else
          lbsa.lbsa_select(lbsa.lbsa_score(q, k, 64, mode="meanpool"), 64, 0.3, "head") if scope == "head" else
          lbsa.lbsa_select_routed(scores, 64, 0.5, 2.0, 2)[0] if scope == "routed" else
          lbsa.lbsa_select_rule(scores, 64, "local_topk", n_valid=500, k=2))
    out, lse = lbsa.lbsa_attend(q, k, v, bs, want_lse=True)
    got = lbsa.lbsa_attend_backward(q, k, v, bs, out, lse, dout)
    rp, col = gpu_csr(bs)
    keep = np.zeros((3 * 8, 8), dtype=bool)
    for r, cols in enumerate(oracle.csr_rows(rp, col)):
        keep[r, cols] = True
    ref, bounds = _reference(q, k, v, dout, _pairs(keep.reshape(1, 3, 8, 8), 500, 64, False), dtype)
    want = oracle.sparse_attention_grad(*(host(x) for x in (q, k, v, dout)), 500, 64, rp, col)
    for a, b in zip(ref, want):
        assert np.allclose(a, b, atol=1e-12)              # this file's dense reference is the oracle's
    _check(got, ref, bounds)


def test_against_differences_of_the_forward_oracle():
    B, H, N, d, block = 1, 1, 150, 64, 64
    keep = _keep(9, B, H, 3, 3, 0.7)
    q, k, v, dout = (_normal(90 + i, B, H, N, d) for i in range(4))
    bs = _blockset(keep, block)
    out, lse = lbsa.lbsa_attend(q, k, v, bs, want_lse=True)
    got = [host(g).astype(np.float64) for g in lbsa.lbsa_attend_backward(q, k, v, bs, out, lse, dout)]
    _, bounds = _reference(q, k, v, dout, _pairs(keep, N, block, False), torch.float32)
    rp, col = gpu_csr(bs)
    x = [host(t).astype(np.float64) for t in (q, k, v)]
    rng, step = np.random.default_rng(1), 1e-4

    def loss(*at):
        return float((oracle.sparse_attention(*at, N, block, rp, col)[0][:, :, :N] * host(dout)).sum())
    for i in range(3):
        u = rng.standard_normal(x[i].shape)
        ends = [loss(*(x[j] + (sign * step * u if j == i else 0) for j in range(3))) for sign in (1, -1)]
        slope = (ends[0] - ends[1]) / (2 * step)
        # second-order differences: step^2 times third derivatives of order |u|^3, far below 1e-4 of the slope's size
        assert abs((got[i] * u).sum() - slope) <= (bounds[i] * np.abs(u)).sum() + 1e-4 * np.linalg.norm(got[i])


def test_bad_block_ids_are_skipped_and_reported():
    q, k, v, dout = (_normal(100 + i, 1, 1, 192, 64, dtype=torch.bfloat16) for i in range(4))
    rp, col = torch.tensor([0, 2, 4, 5]).cuda(), torch.tensor([0, 2, 1, 7, 2]).cuda()
    bad = lbsa.lbsa_blockset_from_csr(rp, col, 1, 1, 3, 64)
    lbsa.lbsa_get_status(bad, clear=True)
    keep = np.zeros((1, 1, 3, 3), dtype=bool)
    keep[0, 0, 0, [0, 2]] = keep[0, 0, 1, 1] = keep[0, 0, 2, 2] = True
    good = _blockset(keep, 64)
    out, lse = lbsa.lbsa_attend(q, k, v, good, want_lse=True)
    want = lbsa.lbsa_attend_backward(q, k, v, good, out, lse, dout)
    got = lbsa.lbsa_attend_backward(q, k, v, bad, out, lse, dout)
    assert lbsa.lbsa_get_status(bad, clear=True) == lbsa.LBSA_ERR_BAD_INDEX
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@BOTH
def test_streams_two_calls_at_once_and_captured_graphs(dtype):
    N, keep = 700, _keep(11, 1, 2, 11, 11, 0.5)
    q, k, v, dout = (_normal(110 + i, 1, 2, N, 128, dtype=dtype) for i in range(4))
    bs = _blockset(keep, 64)
    out, lse = lbsa.lbsa_attend(q, k, v, bs, want_lse=True)

    def step():
        return lbsa.lbsa_attend_backward(q, k, v, bs, out, lse, dout)
    want = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    both = []
    for s in streams:
        with torch.cuda.stream(s):
            both.append(step())
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, step()))
    for (g, _), s in zip(graphs, streams):                # at once, each with its own scratch
        with torch.cuda.stream(s):
            for _ in range(3):
                g.replay()
    torch.cuda.synchronize()
    for got in both + [g for _, g in graphs]:
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert lbsa.lbsa_get_status(bs) == 0


def test_layer_gradients_from_the_output_back_to_the_projections():
    """Norm, rotation, block order, attention and back: the operators together."""
    grid, dims, B, H, d = (3, 7, 9), (16, 24, 24), 1, 2, 64
    n, block = 3 * 7 * 9, 64
    x = [_normal(120 + i, B, n, H, d).transpose(1, 2) for i in range(3)]
    w = [1 + 0.2 * _normal(130 + i, d) for i in range(2)] + [None]
    g = _normal(140, B, n, H, d).transpose(1, 2)
    perm = lbsa.lbsa_partition_perm(*grid, "3d", device="cuda")
    pos = dict(table=lbsa.lbsa_rope_table(grid, dims), grid=grid, dims=dims, perm=perm)
    q, k, v = lbsa.lbsa_norm_rope(x, w, **pos)
    bs = lbsa.lbsa_select(lbsa.lbsa_score(q, k, block), block, 0.7, "row")
    out, lse = lbsa.lbsa_attend(q, k, v, bs, want_lse=True)
    dout, = lbsa.lbsa_permute([g], perm)
    dxs, dws = lbsa.lbsa_norm_rope_backward(lbsa.lbsa_attend_backward(q, k, v, bs, out, lse, dout), x, w, **pos)
    assert lbsa.lbsa_device_status() == 0
    # the same layer through torch autograd in 64 bits
    tx = [host(t).astype(np.float64) for t in x]
    tx = [torch.tensor(t, requires_grad=True) for t in tx]
    tw = [torch.tensor(host(t).astype(np.float64), requires_grad=True) for t in w[:2]]
    ang = torch.tensor(oracle.rope_angles(grid, dims, n))
    order = perm.cpu().long()

    def front(t, wt):
        u = torch.nn.functional.rms_norm(t, (d,), eps=1e-6) * wt
        z = torch.view_as_complex(u.unflatten(-1, (-1, 2)).contiguous()) * torch.polar(torch.ones_like(ang), ang)
        return torch.view_as_real(z).flatten(-2)[:, :, order]
    rp, col = gpu_csr(bs)
    nB = -(-n // block)
    keep = np.zeros((B * H * nB, nB), dtype=bool)
    for r, cols in enumerate(oracle.csr_rows(rp, col)):
        keep[r, cols] = True
    m = torch.tensor(_pairs(keep.reshape(B, H, nB, nB), n, block, False))
    z = front(tx[0], tw[0]) @ front(tx[1], tw[1]).transpose(-1, -2) / d ** 0.5
    o = torch.softmax(z.masked_fill(~m, -torch.inf), -1) @ tx[2][:, :, order]
    want = torch.autograd.grad(o, (*tx, *tw), torch.tensor(host(dout).astype(np.float64)))
    for a, b in zip([*dxs, *dws[:2]], want):
        # a chain of fp32 steps, each within the bounds tested above (1e-5 of the gradients' size for the longest)
        assert np.linalg.norm(host(a) - b.numpy()) <= 1e-5 * np.linalg.norm(b.numpy())
