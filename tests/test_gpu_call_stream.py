"""Calls with `stream=`: new tensors come from that stream's memory, so that they
never take a block which work pending on the current stream still uses."""
import pytest
import torch

import block_sparse_attention_16_b200 as lbsa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)
    lbsa.lbsa_device_status(clear=True)
    yield
    torch.cuda.synchronize()
    assert lbsa.lbsa_device_status() == 0


def _stream_of(t):
    """The stream whose memory a tensor lies in."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not a block of the caching allocator")


def _tensors(got):
    if isinstance(got, torch.Tensor):
        return [got]
    return [t for x in got for t in _tensors(x)] if isinstance(got, (list, tuple)) else []


def _calls():
    grid, dims, n, d = (2, 5, 7), (16, 24, 24), 70, 64
    x, g, w = torch.randn(1, 2, n, d, device="cuda"), torch.randn(1, 2, n, d, device="cuda"), torch.ones(d, device="cuda")
    y, table, perm = x.bfloat16(), lbsa.lbsa_rope_table(grid, dims), lbsa.lbsa_partition_perm(*grid, "3d", device="cuda")
    scores, lse = lbsa.lbsa_score(x, x, 64, want_lse=True)
    bs = lbsa.lbsa_select(scores, 64, 0.9, "row")
    out, lse = lbsa.lbsa_attend(x, x, x, bs, want_lse=True)
    pos = dict(table=table, grid=grid, dims=dims, perm=perm)
    return {
        "rope_table": lambda s: lbsa.lbsa_rope_table(grid, dims, stream=s),
        "rope": lambda s: lbsa.lbsa_rope([x, g], **pos, stream=s),
        "norm_rope": lambda s: lbsa.lbsa_norm_rope([x, g], [w, None], **pos, stream=s),
        "norm_rope_backward": lambda s: lbsa.lbsa_norm_rope_backward([g, x], [x, x], [w, None], **pos, stream=s),
        "attend_backward": lambda s: lbsa.lbsa_attend_backward(x, x, x, bs, out, lse, g, stream=s),
        "attend": lambda s: lbsa.lbsa_attend(x, x, x, bs, want_lse=True, stream=s),
        "score": lambda s: lbsa.lbsa_score(x, x, 64, want_lse=True, stream=s),
        "score_attend": lambda s: lbsa.lbsa_score_attend(y, y, y, 64, want_lse=True, stream=s),
        "select_routed": lambda s: lbsa.lbsa_select_routed(scores, 64, 0.9, 0.5, 2, stream=s)[1:],
        "permute": lambda s: lbsa.lbsa_permute([x, g], perm, stream=s),
        "partition_perm": lambda s: lbsa.lbsa_partition_perm(*grid, "3d", device="cuda", stream=s),
        "export": lambda s: lbsa.lbsa_blockset_export(bs, stream=s),
        "export_bitmask": lambda s: lbsa.lbsa_blockset_export_bitmask(bs, stream=s),
    }


@pytest.mark.parametrize("name", ["rope_table", "rope", "norm_rope", "norm_rope_backward", "attend_backward", "attend", "score",
                                  "score_attend", "select_routed", "permute", "partition_perm", "export",
                                  "export_bitmask"])
def test_new_tensors_belong_to_the_stream_of_the_call(name):
    call, side = _calls()[name], torch.cuda.Stream()
    want = _tensors(call(None))
    torch.cuda.synchronize()
    got = _tensors(call(side))
    side.synchronize()
    assert len(got) == len(want) > 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert [_stream_of(t) for t in got] == [side.cuda_stream] * len(got)
    # a stream of another library: an object that has cuda_stream
    other = _tensors(call(type("Handle", (), {"cuda_stream": side.cuda_stream})()))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, want))
