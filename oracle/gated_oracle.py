"""CPU float64 oracle of the gated recurrence, the q/k norm with rotation and the
state slots (test infrastructure only, like ``la2_oracle``).

The gated form is a reading (the pages mention gated linear attention in one line
and give no formula): the recurrence of the inference form with a gate per token
and head, ``KV_t = exp(gate_t) KV_{t-1} + k_t^T v_t``, ``o_t = q_t KV_t``. The
functions here follow that recurrence token by token; the gradients are its
adjoint, ``U_t = q_t^T do_t + exp(gate_{t+1}) U_{t+1}``. ``tests/test_oracle_gated.py``
pins them by the left product, by ``la2_oracle`` at constant gates and by
differences. The rotation is that of the long-context chapter's RoPE section.
"""

from __future__ import annotations

import numpy as np

from .la2_oracle import _f64


def forward_gated(q, k, v, gate) -> np.ndarray:
    """q, k [B,H,N,d], v [B,H,N,dv], log gates [B,H,N]."""
    q, k, v, g = _f64(q), _f64(k), _f64(v), np.exp(_f64(gate))
    B, H, N, d = q.shape
    out = np.zeros(v.shape)
    state = np.zeros((B, H, d, v.shape[3]))
    for t in range(N):
        state = g[:, :, t, None, None] * state + k[:, :, t, :, None] * v[:, :, t, None, :]
        out[:, :, t] = np.einsum("bhc,bhce->bhe", q[:, :, t], state)
    return out


def backward_gated(q, k, v, do, gate):
    """(dq, dk, dv, dgate) of <do, o>, dgate by the log gates."""
    q, k, v, do, g = _f64(q), _f64(k), _f64(v), _f64(do), np.exp(_f64(gate))
    B, H, N, d = q.shape
    states = np.zeros((N + 1, B, H, d, v.shape[3]))  # states[t]: before token t
    for t in range(N):
        states[t + 1] = g[:, :, t, None, None] * states[t] + k[:, :, t, :, None] * v[:, :, t, None, :]
    dq, dk, dv, dgate = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v), np.zeros(g.shape)
    U = np.zeros(states.shape[1:])  # gradient by the state after token t
    for t in reversed(range(N)):
        dq[:, :, t] = np.einsum("bhe,bhce->bhc", do[:, :, t], states[t + 1])
        U = U + q[:, :, t, :, None] * do[:, :, t, None, :]
        dk[:, :, t] = np.einsum("bhe,bhce->bhc", v[:, :, t], U)
        dv[:, :, t] = np.einsum("bhc,bhce->bhe", k[:, :, t], U)
        dgate[:, :, t] = g[:, :, t] * np.einsum("bhce,bhce->bh", states[t], U)
        U = g[:, :, t, None, None] * U
    return dq, dk, dv, dgate


def kv_state_gated(k, v, gate, state) -> np.ndarray:
    """The state after the tokens, from ``state`` [B,H,d,dv] before them."""
    k, v, g, state = _f64(k), _f64(v), np.exp(_f64(gate)), _f64(state).copy()
    for t in range(k.shape[2]):
        state = g[:, :, t, None, None] * state + k[:, :, t, :, None] * v[:, :, t, None, :]
    return state


def _angles(positions, base, rot, sections):
    """[B,N,rot/2] from positions [axes,B,N]."""
    pos = _f64(positions)
    axis = np.repeat(np.arange(len(sections)), sections)
    freq = np.array([float(base) ** (-2.0 * i / rot) for i in range(rot // 2)])
    return np.moveaxis(pos[axis], 0, -1) * freq


def qk_norm_rope(x, w, positions, base, rot, sections, eps, scale) -> np.ndarray:
    """x [B,N,H,d] -> [B,H,N,d]; w [d] or None."""
    x = _f64(x)
    y = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    if w is not None:
        y = y * _f64(w)
    h = rot // 2
    a = _angles(positions, base, rot, sections)[:, :, None]
    z = y.copy()
    z[..., :h] = y[..., :h] * np.cos(a) - y[..., h:rot] * np.sin(a)
    z[..., h:rot] = y[..., :h] * np.sin(a) + y[..., h:rot] * np.cos(a)
    return np.moveaxis(scale * z, 2, 1)


def qk_norm_rope_backward(dy, x, w, positions, base, rot, sections, eps, scale):
    """(dx [B,N,H,d], dw [d]) from dy [B,H,N,d]."""
    x, g = _f64(x), scale * np.moveaxis(_f64(dy), 1, 2)
    h = rot // 2
    a = _angles(positions, base, rot, sections)[:, :, None]
    z = g.copy()
    z[..., :h] = g[..., :h] * np.cos(a) + g[..., h:rot] * np.sin(a)
    z[..., h:rot] = g[..., h:rot] * np.cos(a) - g[..., :h] * np.sin(a)
    r = 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    u = z if w is None else z * _f64(w)
    dx = r * u - r ** 3 * x * np.mean(u * x, -1, keepdims=True)
    return dx, (z * r * x).sum((0, 1, 2))


def state_copy(pool, src, dst) -> np.ndarray:
    old, new = np.asarray(pool), np.array(pool)
    for s, d in zip(src, dst):
        if d >= 0:
            new[d] = old[s] if s >= 0 else 0.0
    return new


def state_compact(pool, live):
    """(pool, moved)"""
    old, new = np.asarray(pool), np.array(pool)
    n = int(sum(bool(x) for x in live))
    moved = np.full(len(live), -1)
    holes = [i for i in range(n) if not live[i]]
    for i, on in enumerate(live):
        if on and i < n:
            moved[i] = i
        elif on:
            moved[i] = holes.pop(0)
            new[moved[i]] = old[i]
    return new, moved
