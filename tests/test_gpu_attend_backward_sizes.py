"""Attention gradients at the sizes that choose a kernel's shape: fp32 rows a
CTA (16 where fewer than 74 CTAs of 64 rows would run, 32 below 148, else 64),
and bf16 lists long enough for the rings to go round many times.  Bounds as in
test_gpu_attend_backward; bf16 dq's as in test_gpu_attend_backward_keys."""
import numpy as np
import pytest
import torch

import block_sparse_attention_16_b200 as lbsa
from parity import host
from test_gpu_attend_backward import _blockset, _check, _keep, _normal, _pairs, _reference, _run
from test_gpu_attend_backward_keys import _dq_and_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)
    lbsa.lbsa_device_status(clear=True)
    yield
    torch.cuda.synchronize()
    assert lbsa.lbsa_device_status() == 0


# CTAs of 64 rows: 72 and 80 (16 and 32 rows), 144 and 156 (32 and 64), 176 and 352
@pytest.mark.parametrize("per_token", [False, True], ids=["blocks", "tokens"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,N", [(1, 4, 561), (1, 4, 639), (2, 3, 705), (2, 3, 769), (2, 4, 651), (1, 16, 650)])
def test_fp32_rows_of_a_cta(B, H, N, d, per_token):
    nB = -(-N // 64)
    _run(B, H, N, d, 64, torch.float32, _keep(N, B, H, N if per_token else nB, nB, 0.4), per_token, seed=N + d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,N", [(4, 700), (9, 650)])
def test_fp32_blocks_of_128(H, N, d):
    nB = -(-N // 128)
    _run(1, H, N, d, 128, torch.float32, _keep(N, 1, H, nB, nB, 0.6), seed=N + d)


@pytest.mark.parametrize("N,d,block,share,per_token", [
    (4229, 128, 64, 1.0, False), (4160, 64, 64, 0.9, False), (4301, 64, 128, 0.9, False), (4100, 128, 64, 0.5, True),
])
def test_long_lists(N, d, block, share, per_token):
    nB = -(-N // block)
    keep = np.random.default_rng(N).random((1, 1, N if per_token else nB, nB)) < share
    q, k, v, dout = (_normal(N + i, 1, 1, N, d, dtype=torch.bfloat16) for i in range(4))
    bs = _blockset(keep, block, per_token)
    out, lse = lbsa.lbsa_attend(q, k, v, bs, want_lse=True)
    got = lbsa.lbsa_attend_backward(q, k, v, bs, out, lse, dout)
    again = lbsa.lbsa_attend_backward(q, k, v, bs, out, lse, dout)
    assert lbsa.lbsa_get_status(bs) == 0
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    pairs = _pairs(keep, N, block, per_token)
    ref, bounds = _reference(q, k, v, dout, pairs, torch.bfloat16)
    # m: 0 for 64 keys of unit noise, a key of a ragged last piece at most
    last = np.abs(host(k)[:, :, N // 64 * 64:].astype(np.float64)).max(2, keepdims=True) if N % 64 else 0.0
    dq, bound = _dq_and_bound(q, k, v, dout, pairs, last)
    assert np.allclose(dq, ref[0], atol=1e-12)
    _check(got, ref, (bound, *bounds[1:]))
