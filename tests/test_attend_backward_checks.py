"""Refusals of lbsa_attend_backward, before anything is launched (CPU)."""
import ctypes

import pytest
import torch

import block_sparse_attention_16_b200 as lbsa

INV, UNS = lbsa.LBSA_ERR_INVALID_ARG, lbsa.LBSA_ERR_UNSUPPORTED
NAMES = ["q", "k", "v", "out", "dout", "lse", "dq", "dk", "dv"]


def _call(desc=None, bs=None, strides=None, **at):
    # addresses that are never dereferenced: validation fails first
    p = {n: 0x10000 * (i + 1) for i, n in enumerate(NAMES)}
    p.update(at)
    d = dict(B=1, H=2, N_valid=256, d=64, dtype=1, reserved=0, stride_b=2 * 256 * 64, stride_h=256 * 64, stride_n=64)
    d.update(desc or {})
    args = [ctypes.c_void_p(p[n]) for n in NAMES]
    rc = lbsa.load_library().lbsa_attend_backward(*args[:6], ctypes.byref(lbsa._Desc(**d)),
                                                  (ctypes.c_int64 * 24)(*strides) if strides else None, bs, *args[6:], None)
    assert rc == lbsa.LBSA_OK or lbsa.lbsa_last_error()
    return rc


@pytest.mark.parametrize("desc,code", [(dict(d=96), UNS), (dict(N_valid=0), INV), (dict(dtype=7), INV),
                                       (dict(stride_n=60), INV), (dict(stride_n=65), INV), (dict(stride_h=0), INV)])
def test_desc_is_checked(desc, code):
    assert _call(desc) == code


@pytest.mark.parametrize("tensor", range(8))
@pytest.mark.parametrize("at,value", [(0, 0), (1, -64), (2, 32), (2, 66)])
def test_strides_are_checked(tensor, at, value):
    strides = [2 * 256 * 64, 256 * 64, 64] * 8
    strides[3 * tensor + at] = value
    assert _call(dict(B=2), strides=strides) == INV
    assert "stride" in lbsa.lbsa_last_error()


def test_strides_of_single_entries_are_ignored():
    # the batch stride means nothing with B = 1: the call gets as far as the missing blockset
    assert _call(strides=[0, 256 * 64, 64] * 8) == INV
    assert "blockset" in lbsa.lbsa_last_error()


@pytest.mark.parametrize("name", NAMES)
def test_pointers_are_checked(name):
    assert _call(**{name: None}) == INV
    assert name in lbsa.lbsa_last_error()
    assert _call(**{name: 0x90002}) == INV


@pytest.mark.parametrize("a,b", [("dq", "q"), ("dk", "k"), ("dv", "dout"), ("dq", "out"), ("dq", "dk"), ("dk", "dv"),
                                 ("dv", "dq")])
def test_gradients_may_not_alias(a, b):
    assert _call(**{a: 0x10000 * (NAMES.index(b) + 1)}) == INV
    assert "alias" in lbsa.lbsa_last_error()


def test_blockset_is_needed():
    assert _call() == INV
    assert "blockset" in lbsa.lbsa_last_error()


def test_binding_rejects_mismatches():
    q = torch.zeros(1, 1, 64, 64)

    class Set:
        handle = None
    for args in ((q, q, q, Set, q, None, q),                               # no lse
                 (q, q, q, Set, q, torch.zeros(1, 1, 64), q),              # host tensors
                 (q, q, q, Set, q, torch.zeros(1, 1, 64), q.bfloat16()),   # another type
                 (q, q, q, Set, q, torch.zeros(1, 1, 64), q.transpose(2, 3))):
        with pytest.raises(lbsa.LbsaError) as e:
            lbsa.lbsa_attend_backward(*args)
        assert e.value.code == INV
