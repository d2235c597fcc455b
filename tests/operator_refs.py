"""Plain 64-bit forms of the operators around the fold, and the bounds their
fp32 kernels are held to.

Bounds, from the arithmetic and not from any run: u = 2^-24 is half an ulp of
fp32.  A sum of n fp32 products in any order is within 2 (n + 2) u sum|terms|
of the exact one (twice the usual bound, which also covers a tensor core that
truncates where it aligns its products).  The one rounding to the output type
gets no constant: an output has to lie between the roundings of the exact
value less and plus that error.  exp of a rounded difference d is within (|d| + 4) u of the exact one,
relatively (the difference's rounding, and expf's 2 ulp).
"""
from __future__ import annotations

import numpy as np

from lora_moe_expert_gb300 import synth

U = 2.0 ** -24
FLT_MAX = float(np.finfo(np.float32).max)


def sum_bound(n, abs_sum):
    return 2 * (n + 2) * U * abs_sum


def _rne(v, bf16):
    """float64 values rounded to nearest even to the output type (through fp32, which moves a
    value across a bf16 midpoint only from within fp32's own half ulp of it)."""
    with np.errstate(over="ignore"):
        f = np.asarray(v, np.float64).astype(np.float32)
    return (synth.bf16_to_f32(synth.bf16_bits(f)) if bf16 else f).astype(np.float64)


def assert_within(out, ref, err, bf16=False, what=""):
    """out is ref, computed with an error of at most err, then rounded once."""
    out, ref = np.asarray(out, np.float64), np.asarray(ref, np.float64)
    assert out.shape == ref.shape
    assert np.isfinite(out).all(), what
    err = err + U * np.abs(ref) + 1e-37  # fp32's own rounding of the sum
    off = (out < _rne(ref - err, bf16)) | (out > _rne(ref + err, bf16))
    if off.any():
        i = tuple(int(k[0]) for k in np.nonzero(off))
        raise AssertionError(f"{what}: {int(off.sum())} of {out.size} off, first at {i}: "
                             f"{out[i]!r} for {ref[i]!r}, error of {np.broadcast_to(err, out.shape)[i]!r} allowed")


# ---------------------------------------------------------------- router
def route_values(logits):
    """float64 logits, -inf where an expert cannot be chosen."""
    v = np.array(logits, np.float64)
    v[np.isnan(v)] = -np.inf
    return np.minimum(v, FLT_MAX)


def route(logits, top_k, renormalize):
    """(indices, weights, bound of the weights)."""
    v = route_values(logits)
    T, E = v.shape
    idx = np.full((T, top_k), -1, np.int32)
    w = np.zeros((T, top_k))
    bound = np.zeros((T, top_k))
    for t in range(T):
        can = np.flatnonzero(v[t] > -np.inf)
        if can.size == 0:
            continue
        d = v[t] - v[t].max()
        e = np.where(v[t] > -np.inf, np.exp(d), 0.0)
        best = can[np.argsort(-v[t, can], kind="stable")][:top_k]
        z = e[best].sum() if renormalize else e.sum()
        idx[t, :best.size] = best
        w[t, :best.size] = e[best] / z
        # the numerator's, the denominator's (x e^-x <= 0.37 per term) and the quotient's error
        rel = (np.abs(d[best]) + 4 + 0.37 * E + 4 + E + 4) * U
        bound[t, :best.size] = w[t, :best.size] * rel + 2e-38
    return idx, w, bound


def route_loss(logits, indices, dweights, renormalize):
    """sum(weights * dweights) with the chosen experts held fixed."""
    v = route_values(logits)
    total = 0.0
    for t in range(v.shape[0]):
        if not (v[t] > -np.inf).any():
            continue
        e = np.where(v[t] > -np.inf, np.exp(v[t] - v[t].max()), 0.0)
        sel = indices[t] >= 0
        z = e[indices[t][sel]].sum() if renormalize else e.sum()
        total += float((e[indices[t][sel]] / z * dweights[t][sel]).sum())
    return total


def route_grad(logits, indices, weights, dweights, renormalize):
    """(dlogits, bound): the gradient, from the weights as given."""
    v = route_values(logits)
    T, E = v.shape
    K = indices.shape[1]
    grad, mag = np.zeros((T, E)), np.zeros((T, E))
    w, dw = np.asarray(weights, np.float64), np.asarray(dweights, np.float64)
    far = 0.0
    for t in range(T):
        sel = (indices[t] >= 0) & (indices[t] < E)
        at = indices[t][sel]
        s = (w[t][sel] * dw[t][sel]).sum()
        sa = np.abs(w[t][sel] * dw[t][sel]).sum()
        if renormalize:
            p = np.zeros(E)
            p[at] = w[t][sel]
        else:
            can = v[t] > -np.inf
            if can.any():
                d = v[t] - v[t].max()
                e = np.where(can, np.exp(d), 0.0)
                p = e / e.sum()
                far = max(far, np.abs(d[can & (d > -100)]).max())
            else:
                p = np.zeros(E)
        grad[t] = -p * s
        mag[t] = p * sa
        grad[t, at] += w[t][sel] * dw[t][sel]
        mag[t, at] += np.abs(w[t][sel] * dw[t][sel])
    return grad, 2 * (far + 2 * E + K + 16) * U * mag + 2e-38


# ---------------------------------------------------------------- rows
def sort_slots(indices, row_adapter, top_k, n_experts, n_adapters):
    idx = np.asarray(indices, np.int64).reshape(-1)
    cells = n_experts * (n_adapters if row_adapter is not None else 1)
    ok = (idx >= 0) & (idx < n_experts)
    cell = idx.copy()
    if row_adapter is not None:
        s = np.asarray(row_adapter, np.int64)[np.arange(idx.size) // top_k]
        ok &= (s >= 0) & (s < n_adapters)
        cell = s * n_experts + idx
    cell = np.where(ok, cell, cells)
    src = np.argsort(cell, kind="stable")
    pos = np.empty(idx.size, np.int64)
    pos[src] = np.arange(idx.size)
    pos[~ok] = -1
    offsets = np.concatenate([[0], np.cumsum(np.bincount(cell, minlength=cells + 1)[:cells])])
    return offsets.astype(np.int32), src.astype(np.int32), pos.astype(np.int32)


def combine(y, pos, weights, n_tokens, top_k):
    """(out, bound before the rounding); y float64 [n_rows, width]."""
    pos = np.asarray(pos, np.int64).reshape(n_tokens, top_k)
    out, mag = np.zeros((n_tokens, y.shape[1])), np.zeros((n_tokens, y.shape[1]))
    for k in range(top_k):
        there = np.flatnonzero((pos[:, k] >= 0) & (pos[:, k] < y.shape[0]))
        w = 1.0 if weights is None else np.asarray(weights, np.float64)[there, k][:, None]
        row = y[pos[there, k]] * w
        out[there] += row
        mag[there] += np.abs(row)
    return out, sum_bound(top_k, mag)


def combine_grad(dout, y, pos, weights, n_rows, top_k):
    """(dy, named rows, dweights, bound of dweights); dy unrounded, of the named rows."""
    n_tokens = dout.shape[0]
    pos = np.asarray(pos, np.int64).reshape(n_tokens, top_k)
    dy, named = np.zeros((n_rows, dout.shape[1])), np.zeros(n_rows, bool)
    dw, mag = np.zeros((n_tokens, top_k)), np.zeros((n_tokens, top_k))
    for k in range(top_k):
        there = np.flatnonzero((pos[:, k] >= 0) & (pos[:, k] < n_rows))
        r = pos[there, k]
        w = 1.0 if weights is None else np.asarray(weights, np.float64)[there, k][:, None]
        dy[r] = dout[there] * w
        named[r] = True
        if y is not None:
            dw[there, k] = (dout[there] * y[r]).sum(1)
            mag[there, k] = np.abs(dout[there] * y[r]).sum(1)
    return dy, named, dw, sum_bound(dout.shape[1], mag)


# ---------------------------------------------------------------- 4-bit product
def q4_weights(codes, scales, zeros, group):
    """float64 [..., n, k] of codes [..., n, k/2] (low four bits first)."""
    codes = np.asarray(codes)
    q = np.empty(codes.shape[:-1] + (codes.shape[-1] * 2,))
    q[..., 0::2], q[..., 1::2] = codes & 15, codes >> 4
    zero = 8.0 if zeros is None else np.repeat(np.asarray(zeros, np.float64), group, -1)
    return (q - zero) * np.repeat(np.asarray(scales, np.float64), group, -1)


def gather_q4(x, indices, codes, scales, zeros, group, n_slots, top_k):
    """(out, bound before the rounding); x float64 [ceil(n_slots / top_k), k]."""
    E, n = codes.shape[0], codes.shape[1]
    idx = np.zeros(n_slots, np.int64) if indices is None else np.asarray(indices, np.int64)
    out, mag = np.zeros((n_slots, n)), np.zeros((n_slots, n))
    for e in np.unique(idx):
        if 0 <= e < E:
            rows = np.flatnonzero(idx == e)
            w = q4_weights(codes[e], scales[e], None if zeros is None else zeros[e], group)
            out[rows] = x[rows // top_k] @ w.T
            mag[rows] = np.abs(x[rows // top_k]) @ np.abs(w).T
    return out, sum_bound(x.shape[1] + x.shape[1] // group, mag)
