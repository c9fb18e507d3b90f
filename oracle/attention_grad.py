"""Gradients of block-sparse softmax attention in fp64 (oracle; test infrastructure).

For every query row r with kept keys K_r (the valid keys of its kept blocks):
  P = softmax over K_r of scale q_r . k_c,  out_r = sum_c P_c v_c
  dv_c += P_c dout_r,  dP_c = dout_r . v_c,  dS_c = P_c (dP_c - sum_e P_e dP_e)
  dq_r = scale sum_c dS_c k_c,  dk_c += scale dS_c q_r
A row that keeps nothing gives and gets no gradient.
"""
from __future__ import annotations

import numpy as np

from .attention import _f64


def _group_grad(q, k, v, dout, rows, keys, scale, dq, dk, dv):
    z = (q[rows] @ k[keys].T) * scale
    e = np.exp(z - z.max(axis=1, keepdims=True))
    p = e / e.sum(axis=1, keepdims=True)
    dp = dout[rows] @ v[keys].T
    ds = p * (dp - (p * dp).sum(axis=1, keepdims=True))
    dv[keys] += p.T @ dout[rows]
    dq[rows] += scale * (ds @ k[keys])
    dk[keys] += scale * (ds.T @ q[rows])


def sparse_attention_grad(q, k, v, dout, n_valid: int, block: int, row_ptr, col, per_token: bool = False):
    """(dq, dk, dv) [B, H, n_valid, d] of sparse_attention (CSR rows are query
    blocks) or, per_token, of token_sparse_attention (CSR rows are tokens)."""
    q, k, v, dout = (_f64(x)[:, :, :n_valid] for x in (q, k, v, dout))
    B, H, _, d = q.shape
    n_rows = n_valid if per_token else -(-n_valid // block)
    step = 1 if per_token else block
    grads = [np.zeros((B, H, n_valid, d)) for _ in range(3)]
    for b in range(B):
        for h in range(H):
            for i in range(n_rows):
                r = (b * H + h) * n_rows + i
                blocks = np.asarray(col[row_ptr[r]:row_ptr[r + 1]], dtype=np.int64)
                if len(blocks) == 0:
                    continue
                keys = np.concatenate([np.arange(j * block, min((j + 1) * block, n_valid)) for j in blocks])
                rows = np.arange(i * step, min((i + 1) * step, n_valid))
                _group_grad(q[b, h], k[b, h], v[b, h], dout[b, h], rows, keys, 1.0 / np.sqrt(d),
                            *(g[b, h] for g in grads))
    return tuple(grads)
