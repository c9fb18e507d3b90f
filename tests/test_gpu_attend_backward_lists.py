"""Block lists that lbsa_attend_backward cannot answer for, on the GPU."""
import pytest
import torch

import block_sparse_attention_16_b200 as lbsa
from test_gpu_attend_backward import _normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_a_block_named_twice_counts_once_and_is_reported(dtype):
    # the forward pass adds such a block twice: its gradients would not be these
    torch.cuda.set_device(0)
    q, k, v, dout = (_normal(300 + i, 1, 1, 192, 64, dtype=dtype) for i in range(4))

    def lists(rp, col):
        return lbsa.lbsa_blockset_from_csr(torch.tensor(rp).cuda(), torch.tensor(col).cuda(), 1, 1, 3, 64)
    good, bad = lists([0, 2, 4, 5], [0, 2, 1, 2, 2]), lists([0, 3, 5, 7], [0, 0, 2, 1, 2, 2, 2])
    out, lse = lbsa.lbsa_attend(q, k, v, good, want_lse=True)
    want = lbsa.lbsa_attend_backward(q, k, v, good, out, lse, dout)
    assert lbsa.lbsa_get_status(good) == 0
    assert lbsa.lbsa_get_status(bad) == 0
    got = lbsa.lbsa_attend_backward(q, k, v, bad, out, lse, dout)
    assert lbsa.lbsa_get_status(bad, clear=True) == lbsa.LBSA_ERR_BAD_INDEX
    for a, b in zip(got, want):
        assert torch.equal(a, b)
