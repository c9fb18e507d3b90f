"""Refusals of the rotary and norm entry points, before anything is launched (CPU)."""
import ctypes

import pytest
import torch

import block_sparse_attention_16_b200 as lbsa

INV, UNS = lbsa.LBSA_ERR_INVALID_ARG, lbsa.LBSA_ERR_UNSUPPORTED
I3, D3 = ctypes.c_int32 * 3, ctypes.c_double * 3
A = 0x10000                        # addresses that are never dereferenced: validation fails first


def _pos(**kw):
    p = dict(table=A, grid=(2, 3, 4), dims=(16, 24, 24), layout=0)
    p.update(kw)
    return lbsa._RopePos(p["table"], I3(*p["grid"]), I3(*p["dims"]), p["layout"], 0)


def _item(**kw):
    st = (2 * 24 * 64, 24 * 64, 64)
    p = dict(x=A, y=2 * A, dy=3 * A, weight=4 * A, dweight=5 * A, H=2, rotate=1, weight_dtype=1, weight_heads=1,
             x_stride=st, y_stride=st, dy_stride=st)
    p.update(kw)
    for k in ("x_stride", "y_stride", "dy_stride"):
        p[k] = (ctypes.c_int64 * 3)(*p[k])
    return lbsa._RopeItem(**p)


def _call(name, item, pos, count=1, B=1, N=24, d=64, dtype=1, last=1e-6, perm=None):
    lib = lbsa.load_library()
    items = (lbsa._RopeItem * 1)(item) if item is not None else None
    rc = getattr(lib, name)(items, count, B, N, d, dtype, ctypes.byref(pos) if pos is not None else None, perm, last, None)
    assert rc == lbsa.LBSA_OK or lbsa.lbsa_last_error()
    return rc


@pytest.mark.parametrize("kw,code", [
    (dict(table=0), INV), (dict(table=A + 4), INV), (dict(grid=(0, 3, 4)), INV), (dict(grid=(2048, 2048, 512)), INV),
    (dict(dims=(15, 24, 24)), INV), (dict(dims=(-2, 24, 24)), INV), (dict(dims=(0, 0, 0)), INV),
    (dict(dims=(24, 24, 24)), INV), (dict(layout=2), INV), (dict(dims=(8, 8, 8), layout=1), UNS),
])
@pytest.mark.parametrize("name", ["lbsa_norm_rope", "lbsa_norm_rope_backward"])
def test_positions_are_checked(name, kw, code):
    assert _call(name, _item(), _pos(**kw)) == code


@pytest.mark.parametrize("kw", [
    dict(x=0), dict(y=0), dict(x=A + 8), dict(y=A), dict(H=0), dict(weight=4 * A + 4), dict(weight_dtype=2),
    dict(weight_heads=3), dict(x_stride=(2 * 24 * 64, 24 * 64, 32)), dict(y_stride=(2 * 24 * 64, 24 * 64, 66)),
    dict(x_stride=(0, 24 * 64, 64)),
])
@pytest.mark.parametrize("name", ["lbsa_norm_rope", "lbsa_norm_rope_backward"])
def test_tensors_are_checked(name, kw):
    assert _call(name, _item(**kw), _pos(), B=2) == INV


@pytest.mark.parametrize("kw", [dict(dy=0), dict(dy=2 * A), dict(dy=A + 4), dict(dweight=0),
                                dict(dy_stride=(2 * 24 * 64, 24 * 64, 65))])
def test_gradients_are_checked(kw):
    assert _call("lbsa_norm_rope_backward", _item(**kw), _pos()) == INV


@pytest.mark.parametrize("kw,code", [(dict(count=0), INV), (dict(count=4), INV), (dict(B=0), INV), (dict(N=0), INV),
                                     (dict(d=96), UNS), (dict(dtype=2), INV), (dict(B=40000), UNS)])
def test_sizes_are_checked(kw, code):
    assert _call("lbsa_norm_rope", _item(), _pos(), **kw) == code
    assert _call("lbsa_rope", _item(weight=0), _pos(), last=0, **kw) == code


@pytest.mark.parametrize("name,kw", [
    ("lbsa_norm_rope", dict(y=2 * A)), ("lbsa_norm_rope", dict(y=A)), ("lbsa_norm_rope", dict(x=2 * A)),
    ("lbsa_norm_rope_backward", dict(y=2 * A)), ("lbsa_norm_rope_backward", dict(y=A)),
    ("lbsa_norm_rope_backward", dict(y=3 * A)), ("lbsa_norm_rope_backward", dict(x=2 * A)),
    ("lbsa_norm_rope_backward", dict(dy=2 * A)), ("lbsa_norm_rope_backward", dict(dweight=5 * A)),
])
def test_tensors_of_one_call_do_not_alias(name, kw):
    other = dict(x=11 * A, y=12 * A, dy=13 * A, weight=4 * A, dweight=15 * A)
    items = (lbsa._RopeItem * 2)(_item(), _item(**{**other, **kw}))
    rc = getattr(lbsa.load_library(), name)(items, 2, 1, 24, 64, 1, ctypes.byref(_pos()), None, 1e-6, None)
    assert rc == INV and ("alias" in lbsa.lbsa_last_error() or "buffer each" in lbsa.lbsa_last_error())


def test_eps_weight_and_missing_arguments():
    for eps in (-1e-6, float("nan"), float("inf")):
        assert _call("lbsa_norm_rope", _item(), _pos(), last=eps) == INV
        assert _call("lbsa_norm_rope_backward", _item(), _pos(), last=eps) == INV
    assert _call("lbsa_rope", _item(), _pos(), last=0) == INV             # takes no weight
    assert _call("lbsa_rope", _item(weight=0), None, last=0) == INV       # needs positions
    assert _call("lbsa_rope", None, _pos(), last=0) == INV


def test_table_is_checked():
    lib = lbsa.load_library()
    ok = (I3(2, 3, 4), I3(16, 24, 24), 1e4, D3(0, 0, 0), ctypes.c_void_p(A), None)

    def call(**at):
        args = list(ok)
        for i, v in at.items():
            args[int(i[1:])] = v
        return lib.lbsa_rope_table(*args)
    assert call(a0=None) == INV and call(a1=None) == INV and call(a3=None) == INV and call(a4=None) == INV
    for theta in (0.0, -1.0, float("nan"), float("inf")):
        assert call(a2=theta) == INV
    assert call(a3=D3(0, float("nan"), 0)) == INV
    assert call(a0=I3(1, 0, 1)) == INV and call(a1=I3(3, 2, 2)) == INV


def test_binding_rejects_host_tensors_and_mismatches():
    x = torch.zeros(1, 2, 24, 64)
    tab = torch.zeros(224, 2)
    for fn in (lambda: lbsa.lbsa_rope([x], tab, (2, 3, 4), (16, 24, 24)),
               lambda: lbsa.lbsa_norm_rope([x], [torch.ones(64)], tab, (2, 3, 4), (16, 24, 24)),
               lambda: lbsa.lbsa_norm_rope_backward([x], [x], [None]),
               lambda: lbsa.lbsa_norm_rope([x, x], [None]),
               lambda: lbsa.lbsa_norm_rope([], []),
               lambda: lbsa.lbsa_rope([x[0]], tab, (2, 3, 4), (16, 24, 24)),
               lambda: lbsa.lbsa_rope_table((2, 3), (16, 24, 24), table=tab)):
        with pytest.raises(lbsa.LbsaError) as e:
            fn()
        assert e.value.code == INV
    with pytest.raises(lbsa.LbsaError) as e:
        lbsa.lbsa_norm_rope([x.half()], [None])
    assert e.value.code == UNS
