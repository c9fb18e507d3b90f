"""dq of the bf16 attention gradients where keys are far from one another.

dq is summed as sum_c dS_rc (k_c - m), the same number for any m, as
sum_c dS_rc = 0; rounded, it is off by the dS' errors times |k_c - m|.  m is the
mean of 64 keys that the row keeps, 0 where those have little in common, or the
key that it looks at most (one that takes half of the row, or one in a last
piece of fewer than 64).  So keys that a row does not keep, or keeps without a
look at them, must not reach its dq, whatever their size.  Bounds as in
test_gpu_attend_backward, with |k_c| (+ |m| where m need not be 0) in place of
|k_c - m|.
"""
import numpy as np
import pytest
import torch

import block_sparse_attention_16_b200 as lbsa
from parity import host
from test_gpu_attend_backward import E, _blockset, _normal, _pairs

pytestmark = pytest.mark.gpu
H16 = 2.0 ** -8                       # half a step of bf16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)
    lbsa.lbsa_device_status(clear=True)
    yield
    torch.cuda.synchronize()
    assert lbsa.lbsa_device_status() == 0


def _dq_and_bound(q, k, v, dout, pairs, m):
    """dq in fp64 and its bound; m [B, H, N, d]: the most that |m| can be."""
    q, k, v, dout = (host(x).astype(np.float64) for x in (q, k, v, dout))
    (N, d), a, t = q.shape[2:], np.abs, lambda x: x.swapaxes(-1, -2)      # noqa: E731
    scale = d ** -0.5
    z = np.where(pairs, (q @ t(k)) * scale, -np.inf)
    top = np.where(pairs.any(-1, keepdims=True), z.max(-1, keepdims=True), 0.0)
    p = np.exp(z - top)
    l = np.maximum(p.sum(-1, keepdims=True), 1e-300)
    p, lse = p / l, top + np.log(l)
    out, dp = p @ v, dout @ t(v)
    ds = p * (dp - (p * dp).sum(-1, keepdims=True))
    dq = scale * (ds @ k)
    s = np.where(pairs, z, 0.0)
    pe = 4 * E * (a(s) + a(lse) + 4) + d * E * scale * (a(q) @ t(a(k))) + 2.0 ** -13
    oe = (p * (pe + H16)) @ a(v) + (H16 + N * E) * a(out)
    de = (a(dout) * oe).sum(-1, keepdims=True) + d * E * (a(dout) * a(out)).sum(-1, keepdims=True)
    dse = (pe + H16) * a(ds) + p * (de + d * E * (a(dout) @ t(a(v)))) + N * E * a(ds)
    return dq, scale * (dse @ a(k) + dse.sum(-1, keepdims=True) * m) + H16 * a(dq)


def _dq(q, k, v, dout, keep, per_token):
    bs = _blockset(keep, 64, per_token)
    out, lse = lbsa.lbsa_attend(q, k, v, bs, want_lse=True)
    return lbsa.lbsa_attend_backward(q, k, v, bs, out, lse, dout)[0]


def _within(got, want, bound, rows):
    g = host(got).astype(np.float64)[:, :, rows]
    bad = ~(np.abs(g - want[:, :, rows]) <= bound[:, :, rows] + 1e-30)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} off, worst "
                           f"{np.max(np.abs(g - want[:, :, rows]) / (bound[:, :, rows] + 1e-30)):.3g}x of its bound")


def _inputs(seed, N, d):
    return [_normal(seed + i, 1, 2, N, d, dtype=torch.bfloat16) for i in range(4)]


@pytest.mark.parametrize("far", [20.0, 1000.0])
@pytest.mark.parametrize("N,d", [(512, 64), (700, 128)])
@pytest.mark.parametrize("per_token", [False, True], ids=["blocks", "tokens"])
def test_far_keys_that_others_of_the_tile_keep(per_token, N, d, far):
    # even query blocks (tokens) keep even key blocks, odd ones odd: the odd ones' keys lie far away
    q, k, v, dout = _inputs(200, N, d)
    nB = -(-N // 64)
    k = (k.float() + far * _normal(9, d) * (torch.arange(N, device="cuda")[:, None] // 64 % 2)).bfloat16()
    rows = N if per_token else nB
    keep = np.broadcast_to((np.arange(rows)[:, None] + np.arange(nB)) % 2 == 0, (1, 2, rows, nB)).copy()
    mine = np.arange(N) % 2 == 0 if per_token else np.arange(N) // 64 % 2 == 0
    want, bound = _dq_and_bound(q, k, v, dout, _pairs(keep, N, 64, per_token), 0.0)
    _within(_dq(q, k, v, dout, keep, per_token), want, bound, mine)


@pytest.mark.parametrize("share", [1.0, 0.05])
@pytest.mark.parametrize("far", [20.0, 1000.0])
@pytest.mark.parametrize("per_token", [False, True], ids=["blocks", "tokens"])
def test_far_keys_that_a_row_does_not_look_at(per_token, far, share):
    # the first 128 tokens' own keys (or a few of them) point away from every query: logits of -2 |u| far / 8 and less
    N, d = 448, 64
    q, k, v, dout = _inputs(210, N, d)
    u = _normal(8, d)
    n = u.norm()
    q = (q.float() - ((q.float() @ u) / n ** 2 + 4 / n)[..., None] * u).bfloat16()
    on = torch.arange(N, device="cuda") < 128
    on &= torch.arange(N, device="cuda") % 64 < 64 * share
    k = (k.float() - ((k.float() @ u) / n ** 2)[..., None] * u + far * u * on[:, None]).bfloat16()
    keep = np.ones((1, 2, N if per_token else 7, 7), dtype=bool)
    want, bound = _dq_and_bound(q, k, v, dout, _pairs(keep, N, 64, per_token), 0.0)
    _within(_dq(q, k, v, dout, keep, per_token), want, bound, np.arange(N) < N)


@pytest.mark.parametrize("far", [20.0, 1000.0])
@pytest.mark.parametrize("per_token", [False, True], ids=["blocks", "tokens"])
def test_far_keys_in_a_last_piece_of_few(per_token, far):
    # the last piece has three keys, of which no row looks at the last one; some rows keep nothing else
    N, d = 323, 64
    q, k, v, dout = _inputs(230, N, d)
    u = _normal(6, d)
    n = u.norm()
    q = (q.float() - ((q.float() @ u) / n ** 2 + 4 / n)[..., None] * u).bfloat16()
    k[:, :, -1] = far * u
    keep = np.random.default_rng(2).random((1, 2, N if per_token else 6, 6)) < 0.4
    keep[..., 5] = True
    few = np.abs(host(k)[:, :, -3:-1].astype(np.float64)).max(2, keepdims=True)
    want, bound = _dq_and_bound(q, k, v, dout, _pairs(keep, N, 64, per_token), few)
    _within(_dq(q, k, v, dout, keep, per_token), want, bound, np.arange(N) < N)


@pytest.mark.parametrize("far", [1.0, 20.0])
@pytest.mark.parametrize("N", [640, 655])
def test_keys_whose_mean_differs_from_block_to_block(N, far):
    q, k, v, dout = _inputs(220, N, 64)
    nB = -(-N // 64)
    means = far * _normal(7, nB, 64)
    k = (k.float() + means.repeat_interleave(64, 0)[:N]).bfloat16()
    keep = np.random.default_rng(1).random((1, 2, nB, nB)) < 0.5
    keep[:, :, np.arange(nB), np.arange(nB)] = True
    blocks = np.stack([np.abs(host(k)[:, :, i * 64:(i + 1) * 64].astype(np.float64)).max(2) for i in range(nB)], 2)
    most = (blocks[:, :, None] * keep[..., None]).max(3).repeat(64, 2)[:, :, :N]
    want, bound = _dq_and_bound(q, k, v, dout, _pairs(keep, N, 64, False), most)
    _within(_dq(q, k, v, dout, keep, False), want, bound, np.arange(N) < N)
