"""Pins of the sparse-attention gradient oracle: torch autograd through a masked
softmax, differences of the forward oracle, and rows without keys."""
import numpy as np
import pytest
import torch

import oracle


def _case(B, H, N, d, block, per_token, seed):
    rng = np.random.default_rng(seed)
    q, k, v, dout = (rng.standard_normal((B, H, N, d)) for _ in range(4))
    nB = -(-N // block)
    keep = rng.random((B, H, N if per_token else nB, nB)) < 0.5
    keep[0, 0, 1:2] = False
    rp, col = oracle.csr_from_rows([np.nonzero(r)[0] for r in keep.reshape(-1, nB)])
    return (q, k, v, dout), keep, rp, col


@pytest.mark.parametrize("per_token", [False, True])
@pytest.mark.parametrize("B,H,N,d,block", [(2, 2, 37, 8, 8), (1, 1, 16, 4, 16), (1, 3, 50, 6, 16)])
def test_against_autograd_of_a_masked_softmax(B, H, N, d, block, per_token):
    (q, k, v, dout), keep, rp, col = _case(B, H, N, d, block, per_token, 11)
    pairs = np.repeat(keep, block, 3)[..., :N]
    if not per_token:
        pairs = np.repeat(pairs, block, 2)[:, :, :N]
    tq, tk, tv = (torch.tensor(x, requires_grad=True) for x in (q, k, v))
    m = torch.tensor(pairs)
    z = (tq @ tk.transpose(-1, -2) / d ** 0.5).masked_fill(~m, -1e300)
    o = (torch.softmax(z, -1) * m.any(-1, keepdim=True)) @ tv
    want = torch.autograd.grad(o, (tq, tk, tv), torch.tensor(dout))
    got = oracle.sparse_attention_grad(q, k, v, dout, N, block, rp, col, per_token)
    for g, w in zip(got, want):
        assert np.allclose(g, w.numpy(), atol=1e-12)


def test_against_differences_of_the_forward_oracle():
    (q, k, v, dout), keep, rp, col = _case(1, 2, 21, 4, 8, False, 12)
    grads = oracle.sparse_attention_grad(q, k, v, dout, 21, 8, rp, col)

    def loss(q, k, v):
        return float((oracle.sparse_attention(q, k, v, 21, 8, rp, col)[0][:, :, :21] * dout).sum())
    e = 1e-6
    for which in range(3):
        for at in [(0, 0, 0, 0), (0, 1, 9, 2), (0, 1, 20, 3), (0, 0, 12, 1)]:
            up, dn = [x.copy() for x in (q, k, v)], [x.copy() for x in (q, k, v)]
            up[which][at] += e
            dn[which][at] -= e
            assert abs((loss(*up) - loss(*dn)) / (2 * e) - grads[which][at]) < 1e-7


def test_rows_without_keys_and_padding():
    (q, k, v, dout), keep, rp, col = _case(1, 1, 21, 4, 8, False, 13)
    dq, dk, dv = oracle.sparse_attention_grad(q, k, v, dout, 21, 8, rp, col)
    assert not dq[0, 0, 8:16].any()
    padded = [np.concatenate([x, np.full((1, 1, 3, 4), np.nan)], 2) for x in (q, k, v, dout)]
    for g, w in zip(oracle.sparse_attention_grad(*padded, 21, 8, rp, col), (dq, dk, dv)):
        assert np.array_equal(g, w)
