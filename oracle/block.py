"""Reference results of the feed-forward block's operators around the projections (the gated
product, low-rank adapters, the block norms) and of their gradients, by definition, in
float64 numpy.

Test infrastructure (see the package docstring).  Inputs and outputs are plain float64
arrays that hold exactly what the kernels receive.
"""

from __future__ import annotations

import numpy as np

__all__ = ["activation", "gated", "gated_backward", "lora", "lora_backward", "norm", "norm_backward"]

RATE = np.sqrt(2.0 / np.pi)


def _sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def activation(v, name: str):
    """(act(v), act'(v))."""
    if name == "relu":
        return np.where(v > 0, v, 0.0), np.where(v > 0, 1.0, 0.0)
    if name == "silu":
        return v * _sigmoid(v), _sigmoid(v) * (1.0 + v * _sigmoid(-v))
    z = 2.0 * RATE * (v + 0.044715 * v ** 3)  # 0.5 (1 + tanh(z / 2)) = sigmoid(z)
    return v * _sigmoid(z), _sigmoid(z) * (1.0 + v * _sigmoid(-z) * 2.0 * RATE * (1.0 + 3 * 0.044715 * v ** 2))


def gated(w, x, alpha, alpha_up, addend, act: str):
    """(out, pre, bound): pre = [g, u], and the sums of magnitudes behind both."""
    f = w.shape[0] // 2
    rate = np.concatenate([np.full(f, alpha), np.full(f, alpha_up)])
    pre, bound = (x @ w.T) * rate, (np.abs(x) @ np.abs(w).T) * np.abs(rate)
    if addend is not None:
        pre, bound = pre + addend, bound + np.abs(addend)
    return activation(pre[:, :f], act)[0] * pre[:, f:], pre, bound


def gated_backward(grad_out, pre, act: str):
    f = pre.shape[1] // 2
    val, slope = activation(pre[:, :f], act)
    return np.concatenate([grad_out * pre[:, f:] * slope, grad_out * val], 1)


def _groups(a_offsets, ids, t, adapters):
    for z, l in enumerate(np.asarray(ids)):
        b, e = min(int(a_offsets[z]), t), min(int(a_offsets[z + 1]), t)
        if e > b:
            yield slice(b, e), int(l) if 0 <= l < adapters else -1


def lora(x, a, b, a_offsets, ids, scale, base, n: int):
    """(out, z, bound of out's products, bound of z, written): written marks the rows of groups."""
    t, r = x.shape[0], a.shape[1]
    out, bound = np.zeros((t, n)) if base is None else base.copy(), np.zeros((t, n))
    z, zbound, written = np.zeros((t, r)), np.zeros((t, r)), np.zeros(t, bool)
    for rows, l in _groups(a_offsets, ids, t, a.shape[0]):
        written[rows] = True
        if l >= 0:
            z[rows], zbound[rows] = x[rows] @ a[l].T, np.abs(x[rows]) @ np.abs(a[l]).T
            out[rows] += scale[l] * (z[rows] @ b[l].T)
            bound[rows] = np.abs(scale[l]) * (zbound[rows] @ np.abs(b[l]).T)
    return out, z, bound, zbound, written


def lora_backward(grad_out, x, z, a, b, a_offsets, ids, scale, base):
    """(grad_x, grad_a, grad_b, and the sums of magnitudes behind each's products)."""
    t = x.shape[0]
    gx, xb = np.zeros(x.shape) if base is None else base.copy(), np.zeros(x.shape)
    ga, ab, gb, bb = np.zeros(a.shape), np.zeros(a.shape), np.zeros(b.shape), np.zeros(b.shape)
    for rows, l in _groups(a_offsets, ids, t, a.shape[0]):
        if l >= 0:
            s = scale[l]
            dz, zb = grad_out[rows] @ b[l], np.abs(grad_out[rows]) @ np.abs(b[l])
            gx[rows] += s * (dz @ a[l])
            xb[rows] = np.abs(s) * (zb @ np.abs(a[l]))
            ga[l] += s * (dz.T @ x[rows])
            ab[l] += np.abs(s) * (zb.T @ np.abs(x[rows]))
            gb[l] += s * (grad_out[rows].T @ z[rows])
            bb[l] += np.abs(s) * (np.abs(grad_out[rows]).T @ np.abs(z[rows]))
    return gx, ga, gb, xb, ab, bb


def _root(x, eps):
    return np.sqrt((x * x).mean(1, keepdims=True) + eps)


def norm(residual, weight, block, block_weight, gate, scale: float, eps: float, stored):
    """(out, residual_out before it is stored); stored: rounds residual_out to its type."""
    r = residual
    if block is not None:
        p = block if block_weight is None else block / _root(block, eps) * block_weight
        g = 1.0 if gate is None else np.repeat(gate, len(r) // len(gate), 0)
        r = scale * residual + g * p
    held = stored(r)
    return held / _root(held, eps) * weight, r


def norm_backward(grad_out, grad_res, res, weight, block, block_weight, gate, scale: float, eps: float):
    """The gradients by name, and for each the sum of magnitudes behind it (key + "_bound")."""
    t, h = res.shape
    root = _root(res, eps)
    unit, a = res / root, grad_out * weight
    along = (a * unit).mean(1, keepdims=True)
    d = (a - unit * along) / root + (0.0 if grad_res is None else grad_res)
    size = (np.abs(a) + np.abs(unit) * (np.abs(a * unit)).mean(1, keepdims=True)) / root
    size = size + (0.0 if grad_res is None else np.abs(grad_res))
    scale = 1.0 if block is None else scale
    out = {"residual": scale * d, "residual_bound": abs(scale) * size, "weight": (grad_out * unit).sum(0),
           "weight_bound": np.abs(grad_out * unit).sum(0)}
    if block is None:
        return out
    per = 1 if gate is None else t // len(gate)
    g = np.ones((1, h)) if gate is None else np.repeat(gate, per, 0)
    p = block
    if block_weight is not None:
        root_o = _root(block, eps)
        unit_o = block / root_o
        b, bs = d * g * block_weight, size * np.abs(g * block_weight)
        out["block"] = (b - unit_o * (b * unit_o).mean(1, keepdims=True)) / root_o
        out["block_bound"] = (bs + np.abs(unit_o) * (bs * np.abs(unit_o)).mean(1, keepdims=True)) / root_o
        out["block_weight"] = (d * g * unit_o).sum(0)
        out["block_weight_bound"] = (size * np.abs(g * unit_o)).sum(0)
        p = unit_o * block_weight
    else:
        out["block"], out["block_bound"] = d * g, size * np.abs(g)
    if gate is not None:
        out["gate"] = (d * p).reshape(len(gate), per, h).sum(1)
        out["gate_bound"] = (size * np.abs(p)).reshape(len(gate), per, h).sum(1)
    return out
