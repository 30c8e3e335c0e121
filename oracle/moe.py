"""Reference results of the int4 linear layer and of the mixture-of-experts
operators around the grouped products, by definition, in float64 numpy.

Test infrastructure (see the package docstring).  Inputs and outputs are plain
values: codes as integers, activations and logits as float64 arrays that hold
exactly what the kernels receive.
"""

from __future__ import annotations

import numpy as np

__all__ = ["int4_dequant", "int4_linear", "int4_grouped", "route", "route_backward", "sort", "gather", "combine",
           "combine_backward", "swiglu", "swiglu_backward"]


def int4_dequant(packed, scale, zero, k: int, group: int) -> np.ndarray:
    """D[n, k] = (code - zero) * scale of uint8 [N, (K + 1) / 2] codes (even k in the low
    nibble), scale [N, G] and zero [N, G] or None (8)."""
    p = np.asarray(packed, np.uint8)
    codes = np.empty((p.shape[0], 2 * p.shape[1]))
    codes[:, 0::2] = p & 15
    codes[:, 1::2] = p >> 4
    g = np.arange(k) // group
    z = 8.0 if zero is None else np.asarray(zero, np.float64)[:, g]
    return (codes[:, :k] - z) * np.asarray(scale, np.float64)[:, g]


def int4_linear(packed, scale, zero, x, group: int):
    """(x @ D^T, bound): the bound is sum_k |x| (code + zero) |scale|, what the grouped
    evaluation scale * (sum x code - zero * sum x) can be off by per unit of rounding."""
    x = np.asarray(x, np.float64)
    k = x.shape[1]
    d = int4_dequant(packed, scale, zero, k, group)
    ones = np.abs(np.asarray(scale, np.float64))
    size = int4_dequant(packed, ones, np.zeros_like(ones), k, group)
    z = np.full(ones.shape, 8.0) if zero is None else np.asarray(zero, np.float64)
    size = size + (z * ones)[:, np.arange(k) // group]
    return x @ d.T, np.abs(x) @ size.T


def int4_grouped(packed, scale, zero, x, group: int, a_offsets, expert_ids):
    """(out, bound, written): rows a_offsets[z] .. a_offsets[z + 1] - 1 times expert
    expert_ids[z] (outside 0 .. E - 1: zeros); written marks the rows some group covers."""
    t, n, e = x.shape[0], packed.shape[1], packed.shape[0]
    out, bound, written = np.zeros((t, n)), np.zeros((t, n)), np.zeros(t, bool)
    for z, ex in enumerate(np.asarray(expert_ids)):
        b, c = min(int(a_offsets[z]), t), min(int(a_offsets[z + 1]), t)
        if c <= b:
            continue
        written[b:c] = True
        if 0 <= ex < e:
            out[b:c], bound[b:c] = int4_linear(packed[ex], scale[ex], None if zero is None else zero[ex], x[b:c], group)
    return out, bound, written


def route(logits, top_k: int, renormalize: bool):
    """(ids, weights) of the top_k logits of every row, largest first, the lower index
    first among equals, -inf and NaN never; softmax over the chosen or over all."""
    t, e = logits.shape
    ids, weights = np.full((t, top_k), -1, np.int32), np.zeros((t, top_k))
    for i, row in enumerate(np.asarray(logits, np.float64)):
        able = [j for j in range(e) if row[j] > -np.inf]
        pick = sorted(able, key=lambda j: (-row[j], j))[:top_k]
        ids[i, :len(pick)] = pick
        if np.isnan(row).any():
            weights[i] = np.nan
        elif pick:
            pool = row[pick] if renormalize else row
            with np.errstate(invalid="ignore"):
                weights[i, :len(pick)] = np.exp(row[pick] - row[pick[0]]) / np.exp(pool - row[pick[0]]).sum()
    return ids, weights


def route_backward(logits, ids, grad_weights, renormalize: bool):
    """Gradient of route's weights with respect to the logits (ids are constants)."""
    row = np.asarray(logits, np.float64)
    t, e = row.shape
    a, chosen = np.zeros((t, e)), np.zeros((t, e), bool)
    for i in range(t):
        for j, ex in enumerate(ids[i]):
            if 0 <= ex < e:
                a[i, ex] += grad_weights[i, j]
                chosen[i, ex] = True
    out = np.zeros((t, e))
    for i in range(t):
        pool = chosen[i] if renormalize else row[i] > -np.inf
        if pool.any():
            p = np.where(pool, np.exp(np.where(pool, row[i] - row[i][pool].max(), 0.0)), 0.0)
            p /= p.sum()
            out[i] = p * (a[i] - (p * a[i]).sum())
    return out


def sort(expert_ids, num_experts: int):
    """(a_offsets, row_slot, slot_row) of a stable sort by expert, ids outside
    0 .. num_experts - 1 last and complemented."""
    flat = np.asarray(expert_ids).reshape(-1).astype(np.int64)
    key = np.where((flat < 0) | (flat >= num_experts), num_experts, flat)
    order = np.argsort(key, kind="stable")
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=num_experts + 1))])[:num_experts + 1]
    dropped = key[order] == num_experts
    row = np.arange(flat.size)
    slot_row = np.empty(flat.size, np.int64)
    slot_row[order] = np.where(dropped, ~row, row)
    return offsets, np.where(dropped, ~order, order), slot_row.reshape(np.asarray(expert_ids).shape)


def gather(x, slot_row):
    out = np.zeros((slot_row.size, x.shape[1]))
    for (t, _), r in np.ndenumerate(slot_row):
        out[r if r >= 0 else ~r] = x[t] if r >= 0 else 0.0
    return out


def combine(rows, slot_row, weights):
    """(out, bound): the weighted sum over live slots, and the sum of magnitudes."""
    t, _ = slot_row.shape
    out, bound = np.zeros((t, rows.shape[1])), np.zeros((t, rows.shape[1]))
    for (i, j), r in np.ndenumerate(slot_row):
        if r >= 0:
            w = 1.0 if weights is None else float(weights[i, j])
            out[i] += w * rows[r]
            bound[i] += np.abs(w * rows[r])
    return out, bound


def combine_backward(grad_out, rows, slot_row, weights):
    """(grad_rows, grad_weights, bound of grad_weights)."""
    gr = np.zeros(rows.shape)
    gw, bound = np.zeros(slot_row.shape), np.zeros(slot_row.shape)
    for (i, j), r in np.ndenumerate(slot_row):
        if r >= 0:
            gr[r] = float(weights[i, j]) * grad_out[i]
            gw[i, j] = grad_out[i] @ rows[r]
            bound[i, j] = np.abs(grad_out[i]) @ np.abs(rows[r])
    return gr, gw, bound


def _sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def swiglu(x):
    f = x.shape[1] // 2
    g, u = x[:, :f], x[:, f:]
    return g * _sigmoid(g) * u


def swiglu_backward(grad_y, x):
    """(grad_x, bound): the bound is the gradient with |1| + |g (1 - sig)| for 1 + g (1 - sig)."""
    f = x.shape[1] // 2
    g, u = x[:, :f], x[:, f:]
    s, rest = _sigmoid(g), _sigmoid(-g)
    dg, du = grad_y * u * s * (1.0 + g * rest), grad_y * g * s
    return np.concatenate([dg, du], 1), np.concatenate([np.abs(grad_y * u * s) * (1.0 + np.abs(g) * rest), np.abs(du)], 1)
