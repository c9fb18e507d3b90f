"""Pins of the rotary and norm oracle: complex arithmetic, torch autograd,
differences, and the properties of a rotation."""
import numpy as np
import pytest
import torch

import oracle

GRID, DIMS = (3, 4, 5), (4, 6, 2)


def _rows(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


def test_angles_by_hand():
    a = oracle.rope_angles((2, 2, 2), (2, 4, 2), 9, theta=100.0, start=(5, 0, 1))
    assert a.shape == (9, 4)
    assert np.allclose(a[0], [5, 0, 0, 1])
    assert np.allclose(a[7], [6, 1, 0.1, 2])       # t = h = w = 1; second height frequency 100^(-1/2)
    assert not a[8].any()                          # past the grid


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rotation_is_complex_multiplication(layout):
    n, d, rd = 60, 16, sum(DIMS)
    x, ang = _rows(1, 2, 3, n, d), oracle.rope_angles(GRID, DIMS, n)
    y = oracle.rope_rotate(x, ang, layout)
    head = x[..., :rd]
    z = head[..., 0::2] + 1j * head[..., 1::2] if layout == "interleaved" else head[..., :rd // 2] + 1j * head[..., rd // 2:]
    z = z * np.exp(1j * ang)
    want = x.copy()
    if layout == "interleaved":
        want[..., 0:rd:2], want[..., 1:rd:2] = z.real, z.imag
    else:
        want[..., :rd // 2], want[..., rd // 2:rd] = z.real, z.imag
    assert np.allclose(y, want, atol=1e-13)
    assert np.allclose(oracle.rope_rotate(y, ang, layout, inverse=True), x, atol=1e-13)


def test_scores_depend_on_differences_of_positions():
    q, k = _rows(2, 1, 1, 1, 12).repeat(60, 2), _rows(3, 1, 1, 1, 12).repeat(60, 2)
    ang = oracle.rope_angles(GRID, DIMS, 60)
    s = (oracle.rope_rotate(q, ang) @ oracle.rope_rotate(k, ang).swapaxes(-1, -2))[0, 0]
    tok = np.arange(60).reshape(GRID)
    for a, b in (((0, 0, 0), (1, 2, 3)), ((1, 1, 1), (2, 3, 4))):
        assert np.isclose(s[tok[a], tok[b]], s[tok[0, 1, 1], tok[1, 3, 4]])


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("per_head", [False, True])
def test_norm_rope_and_its_gradient_against_autograd(layout, per_head):
    B, H, n, d = 2, 3, 61, 16
    x, dy = _rows(4, B, H, n, d), _rows(5, B, H, n, d)
    w = 1 + 0.3 * (_rows(6, H, d) if per_head else _rows(6, d))
    ang = oracle.rope_angles(GRID, DIMS, n)
    tx, tw = torch.tensor(x, requires_grad=True), torch.tensor(w, requires_grad=True)
    u = torch.nn.functional.rms_norm(tx, (d,), eps=1e-6) * (tw[:, None] if per_head else tw)
    m = np.stack([oracle.rope_rotate(np.eye(d), np.repeat(ang[t:t + 1], d, 0), layout) for t in range(n)])   # row @ m[t]
    y = torch.einsum("bhnd,nde->bhne", u, torch.tensor(m))
    assert np.allclose(oracle.norm_rope(x, w, ang, layout), y.detach().numpy(), atol=1e-12)
    gx, gw = torch.autograd.grad(y, (tx, tw), torch.tensor(dy))
    dx, dw = oracle.norm_rope_grad(dy, x, w, ang, layout)
    assert np.allclose(dx, gx.numpy(), atol=1e-11)
    assert dw.shape == w.shape and np.allclose(dw, gw.numpy(), atol=1e-10)


def test_norm_rope_gradient_against_differences():
    x, dy, w = _rows(7, 1, 2, 4, 12), _rows(8, 1, 2, 4, 12), 1 + 0.2 * _rows(9, 12)
    ang = oracle.rope_angles((2, 1, 2), (4, 4, 4), 4)
    dx, dw = oracle.norm_rope_grad(dy, x, w, ang)
    loss = lambda a, b: float((oracle.norm_rope(a, b, ang) * dy).sum())     # noqa: E731
    e = 1e-6
    for at in [(0, 0, 0, 0), (0, 1, 3, 7), (0, 1, 2, 11)]:
        up, dn = x.copy(), x.copy()
        up[at] += e
        dn[at] -= e
        assert abs((loss(up, w) - loss(dn, w)) / (2 * e) - dx[at]) < 1e-7
    for at in (0, 5, 11):
        up, dn = w.copy(), w.copy()
        up[at] += e
        dn[at] -= e
        assert abs((loss(x, up) - loss(x, dn)) / (2 * e) - dw[at]) < 1e-7
