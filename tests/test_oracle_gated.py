"""Pins of the gated form, the q/k norm with rotation and the slot moves in the
float64 oracle: the left product with its decay matrix, the plain and the decayed
op at constant gates, restarts against separate sequences, and differences."""

import numpy as np
import pytest

import oracle


def _rand(*shape, seed=0):
    return np.random.default_rng(seed).standard_normal(shape)


def _inputs(B, H, N, d, dv, seed):
    return (_rand(B, H, N, d, seed=seed), _rand(B, H, N, d, seed=seed + 1), _rand(B, H, N, dv, seed=seed + 2),
            -np.abs(_rand(B, H, N, seed=seed + 3)))


def test_forward_is_the_left_product():
    q, k, v, g = _inputs(2, 2, 9, 3, 4, 1)
    c = np.cumsum(g, -1)
    D = np.tril(np.exp(c[..., :, None] - c[..., None, :]))
    ref = ((q @ np.swapaxes(k, -1, -2)) * D) @ v
    assert np.allclose(oracle.forward_gated(q, k, v, g), ref, rtol=1e-12, atol=1e-12)


def test_hand_example():
    # gates 1/2 and 1/4 before tokens 1 and 2: o_1 = 2 (1/2 + 2) = 5, o_2 = 3 (1/8 + 2/4 + 4) = 13.875
    q = np.array([1.0, 2.0, 3.0]).reshape(1, 1, 3, 1)
    k, v = np.ones((1, 1, 3, 1)), np.array([1.0, 2.0, 4.0]).reshape(1, 1, 3, 1)
    g = np.log(np.array([0.7, 0.5, 0.25])).reshape(1, 1, 3)
    assert np.allclose(oracle.forward_gated(q, k, v, g)[0, 0, :, 0], [1.0, 5.0, 13.875], rtol=1e-14)


@pytest.mark.parametrize("lam", [1.0, 0.9, 0.3])
def test_constant_gates_are_the_decayed_op(lam):
    q, k, v, g = _inputs(1, 2, 11, 4, 3, 5)
    do = _rand(1, 2, 11, 3, seed=9)
    g = np.full_like(g, np.log(lam))
    assert np.allclose(oracle.forward_gated(q, k, v, g), oracle.forward_decay(q, k, v, [lam, lam]), atol=1e-12)
    for a, b in zip(oracle.backward_gated(q, k, v, do, g), oracle.backward_decay(q, k, v, do, [lam, lam])):
        assert np.allclose(a, b, atol=1e-12)


def test_restart_separates_documents():
    q, k, v, g = _inputs(1, 1, 10, 3, 3, 8)
    do = _rand(1, 1, 10, 3, seed=4)
    g[..., 6] = -np.inf
    whole = oracle.backward_gated(q, k, v, do, g)
    assert np.allclose(oracle.forward_gated(q, k, v, g)[:, :, 6:],
                       oracle.forward_gated(q[:, :, 6:], k[:, :, 6:], v[:, :, 6:], g[:, :, 6:]), atol=1e-13)
    part = oracle.backward_gated(q[:, :, :6], k[:, :, :6], v[:, :, :6], do[:, :, :6], g[:, :, :6])
    for a, b in zip(whole, part):
        assert np.allclose(a[:, :, :6], b, atol=1e-13)
    assert whole[3][0, 0, 6] == 0.0


def test_gradients_by_differences():
    q, k, v, g = _inputs(1, 2, 7, 3, 2, 21)
    do = _rand(1, 2, 7, 2, seed=33)
    grads = oracle.backward_gated(q, k, v, do, g)
    for i in range(4):
        step = _rand(*(q, k, v, g)[i].shape, seed=50 + i)

        def loss(e):
            x = [q, k, v, g]
            x[i] = x[i] + e * step
            return float((oracle.forward_gated(*x) * do).sum())

        # central differences with h = 1e-4: error h^2 f''' / 6, below 1e-6 here
        num = (loss(1e-4) - loss(-1e-4)) / 2e-4
        assert abs(num - float((grads[i] * step).sum())) <= 1e-6 * max(1.0, abs(num))


def test_state_continues_the_forward():
    q, k, v, g = _inputs(1, 2, 12, 3, 4, 2)
    ref = oracle.forward_gated(q, k, v, g)
    s = oracle.kv_state_gated(k[:, :, :7], v[:, :, :7], g[:, :, :7], np.zeros((1, 2, 3, 4)))
    for t in range(7, 12):
        s = oracle.kv_state_gated(k[:, :, t:t + 1], v[:, :, t:t + 1], g[:, :, t:t + 1], s)
        assert np.allclose(np.einsum("bhc,bhce->bhe", q[:, :, t], s), ref[:, :, t], atol=1e-12)


def _pos(B, N, axes, seed=0):
    return np.random.default_rng(seed).integers(0, 50, (axes, B, N))


def test_rotation_keeps_relative_positions():
    """Without a weight, <z_q, z_k> depends on the difference of the positions only."""
    x, y = _rand(1, 1, 1, 8, seed=1), _rand(1, 1, 1, 8, seed=2)
    dots = []
    for a, b in ((3, 10), (103, 110), (0, 7)):
        u = oracle.qk_norm_rope(x, None, np.full((1, 1, 1), a), 100.0, 8, (4,), 0.0, 1.0)
        v = oracle.qk_norm_rope(y, None, np.full((1, 1, 1), b), 100.0, 8, (4,), 0.0, 1.0)
        dots.append(float((u * v).sum()))
    assert np.allclose(dots, dots[0], rtol=1e-12)


def test_norm_and_unrotated_tail():
    x = _rand(2, 3, 2, 10, seed=5)
    z = oracle.qk_norm_rope(x, None, _pos(2, 3, 1), 10.0, 6, (3,), 0.0, 2.0)
    assert np.allclose((z * z).mean(-1), 4.0)
    y = np.moveaxis(x / np.sqrt((x * x).mean(-1, keepdims=True)), 2, 1)
    assert np.allclose(z[..., 6:], 2.0 * y[..., 6:])
    # a pair on an axis whose position is 0 does not turn
    pos = np.stack([np.zeros((2, 3)), np.ones((2, 3))])
    z = oracle.qk_norm_rope(x, None, pos, 10.0, 6, (1, 2), 0.0, 1.0)
    assert np.allclose(z[..., [0, 3]], y[..., [0, 3]]) and not np.allclose(z[..., 1], y[..., 1])


def test_rope_gradients_by_differences():
    x, w, dy = _rand(2, 3, 2, 8, seed=1), _rand(8, seed=2), _rand(2, 2, 3, 8, seed=3)
    args = (_pos(2, 3, 3), 10.0, 6, (1, 1, 1), 1e-3, 0.7)
    dx, dw = oracle.qk_norm_rope_backward(dy, x, w, *args)
    for grad, which in ((dx, 0), (dw, 1)):
        step = _rand(*grad.shape, seed=11 + which)

        def loss(e):
            a, b = (x + e * step, w) if which == 0 else (x, w + e * step)
            return float((oracle.qk_norm_rope(a, b, *args) * dy).sum())

        num = (loss(1e-4) - loss(-1e-4)) / 2e-4
        assert abs(num - float((grad * step).sum())) <= 1e-6 * max(1.0, abs(num))


def test_slot_moves():
    pool = np.arange(6.0)[:, None]
    assert oracle.state_copy(pool, [0, 0, -1], [2, 3, 5])[:, 0].tolist() == [0, 1, 0, 0, 4, 0]
    new, moved = oracle.state_compact(pool, [0, 1, 0, 1, 1, 0])
    assert moved.tolist() == [-1, 1, -1, 0, 2, -1]
    assert new[:3, 0].tolist() == [3, 1, 4]
