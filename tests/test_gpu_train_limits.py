"""Far offsets and the largest block counts of the rotary, norm and attention
gradient kernels: the same bits as a compact call, or the oracle's rows."""
import numpy as np
import pytest
import torch

import oracle
import block_sparse_attention_16_b200 as lbsa

pytestmark = pytest.mark.gpu
FAR = 2 ** 31 + 64                      # elements between the two batch entries


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)
    lbsa.lbsa_device_status(clear=True)
    yield
    torch.cuda.synchronize()
    assert lbsa.lbsa_device_status() == 0
    torch.cuda.empty_cache()


def _normal(seed, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


def _apart(shape, dtype, count):
    """`count` tensors of the shape whose batch entries lie FAR elements apart, in one buffer."""
    B, H, N, d = shape
    assert B == 2
    one = H * N * d
    buf = torch.empty(FAR + count * one, dtype=dtype, device="cuda")
    return [buf.as_strided(shape, (FAR, N * d, d, 1), i * one) for i in range(count)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_offsets_past_32_bits(dtype):
    shape = (2, 2, 200, 64)
    near = [_normal(i, *shape, dtype=dtype) for i in range(5)]
    far = _apart(shape, dtype, 11)
    for a, b in zip(near, far):
        b.copy_(a)
    rp, col = torch.tensor([0, 2, 3, 4, 6] + [0] * 12).cuda(), torch.tensor([0, 2, 1, 3, 0, 1] * 4).cuda()
    rp = torch.cat([torch.tensor([0]).cuda(), (rp[1:5].repeat(4) + torch.arange(4).cuda().repeat_interleave(4) * 6)])
    bs = lbsa.lbsa_blockset_from_csr(rp, col, 2, 2, 4, 64)
    q, k, v, dout, x = near
    out, lse = lbsa.lbsa_attend(q, k, v, bs, want_lse=True)
    far[5].copy_(out)
    want = lbsa.lbsa_attend_backward(q, k, v, bs, out, lse, dout)
    got = lbsa.lbsa_attend_backward(*far[:3], bs, far[5], lse, far[3], *far[6:9])
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    w = 1 + 0.1 * _normal(9, 64, dtype=torch.float32)
    pos = dict(table=lbsa.lbsa_rope_table((5, 5, 8), (16, 24, 24)), grid=(5, 5, 8), dims=(16, 24, 24))
    y, = lbsa.lbsa_norm_rope([x], [w], **pos)
    lbsa.lbsa_norm_rope([far[4]], [w], outs=[far[9]], **pos)
    assert torch.equal(far[9], y)
    (dx,), (dw,) = lbsa.lbsa_norm_rope_backward([dout], [x], [w], **pos)
    _, (fw,) = lbsa.lbsa_norm_rope_backward([far[3]], [far[4]], [w], dxs=[far[10]], **pos)
    assert torch.equal(far[10], dx) and torch.equal(fw, dw)


@pytest.mark.parametrize("block", [64, 128])
def test_the_most_blocks(block):
    # 4,096 blocks, the last one ragged; every query block keeps one near and one far key block
    nB, d = 4096, 64
    N = nB * block - 17
    q, k, v, dout = (_normal(20 + i, 1, 1, N, d) for i in range(4))
    cols = torch.stack([torch.arange(nB), (torch.arange(nB) * 37 + 2000) % nB], 1)
    cols[:, 1] = torch.where(cols[:, 0] == cols[:, 1], (cols[:, 1] + 1) % nB, cols[:, 1])
    cols = cols.sort(1).values
    bs = lbsa.lbsa_blockset_from_csr((torch.arange(nB + 1) * 2).cuda(), cols.reshape(-1).cuda(), 1, 1, nB, block)
    out, lse = lbsa.lbsa_attend(q, k, v, bs, want_lse=True)
    dq, dk, dv = lbsa.lbsa_attend_backward(q, k, v, bs, out, lse, dout)
    assert lbsa.lbsa_get_status(bs) == 0
    # every query and key block that touches key blocks `some`, as a problem of its own
    some = [0, 1, 2047, nB - 1]
    rows = [i for i in range(nB) if set(cols[i].tolist()) & set(some)]
    need = sorted(set(rows) | set(some) | {int(c) for i in rows for c in cols[i]})
    take = torch.cat([torch.arange(j * block, min((j + 1) * block, N)) for j in need]).cuda()
    at = {j: n for n, j in enumerate(need)}
    rp, col = oracle.csr_from_rows([sorted(at[int(c)] for c in cols[j]) if j in rows else [] for j in need])
    sub = [x[:, :, take].float().cpu().numpy() for x in (q, k, v, dout)]
    ref = oracle.sparse_attention_grad(*sub, len(take), block, rp, col)
    spans = np.cumsum([0] + [min((j + 1) * block, N) - j * block for j in need])
    for got, want, blocks in ((dq, ref[0], rows), (dk, ref[1], some), (dv, ref[2], some)):
        for j in blocks:
            a = got[0, 0, j * block:min((j + 1) * block, N)].float().cpu().numpy()
            b = want[0, 0, spans[at[j]]:spans[at[j] + 1]]
            # P, dS, out and the gradient itself rounded to bf16, up to 256 terms of either sign: 4 roundings of 2^-8
            assert np.linalg.norm(a - b) <= 4 * 2.0 ** -8 * np.linalg.norm(b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_values_of_unused_blocks_do_not_matter(dtype):
    # key blocks 4 and 5 (a 128-row tile) are kept by nobody, query blocks 6 and 7 keep nothing
    N, nB = 600, 10
    keep = np.random.default_rng(3).random((1, 2, nB, nB)) < 0.5
    keep[:, :, :, 4:6] = False
    keep[:, :, 6:8] = False
    keep[:, :, 0, 0] = True
    rp, col = oracle.csr_from_rows([np.nonzero(r)[0] for r in keep.reshape(-1, nB)])
    bs = lbsa.lbsa_blockset_from_csr(torch.from_numpy(rp).cuda(), torch.from_numpy(col).cuda(), 1, 2, nB, 64)
    q, k, v, dout = (_normal(40 + i, 1, 2, N, 64, dtype=dtype) for i in range(4))
    out, lse = lbsa.lbsa_attend(q, k, v, bs, want_lse=True)
    want = lbsa.lbsa_attend_backward(q, k, v, bs, out, lse, dout)
    k[:, :, 256:384], v[:, :, 256:384] = float("inf"), float("nan")
    q[:, :, 384:512], dout[:, :, 384:512] = float("nan"), -float("inf")
    got = lbsa.lbsa_attend_backward(q, k, v, bs, out, lse, dout)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert not got[0][:, :, 384:512].any() and not got[1][:, :, 256:384].any() and not got[2][:, :, 256:384].any()
