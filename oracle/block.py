"""Float64 oracle of the operators around the MoE layer: block norms with gate
and residual scale, the global gradient norm with clipping, and low-rank
adapters.  Plain numpy from the formulas, one step per line; test
infrastructure only, sharing no code with the library.

N(v) = v / sqrt(mean_c v_c^2 + eps) along the last axis."""
from __future__ import annotations

import numpy as np


def rms_inv(v, eps):
    return 1.0 / np.sqrt(np.mean(v * v, axis=1, keepdims=True) + eps)


def combine(Y, row_map, w):
    """y[t] = sum_j w[t, j] Y[row_map[t, j]] (w None: ones)."""
    T, k = row_map.shape
    y = np.zeros((T, Y.shape[1]))
    for j in range(k):
        y += (1.0 if w is None else w[:, j:j + 1]) * Y[row_map[:, j]]
    return y


def block_norm_forward(h, y=None, *, w_post=None, gate=None, row_gate=None, res_scale=1.0,
                       w_pre=None, eps=1e-6):
    """(h1 or None, x or None): h1 = a h + row_gate gate N(y) w_post, x = N(h1) w_pre."""
    h1 = h
    if y is not None:
        n = y if w_post is None else y * rms_inv(y, eps) * w_post
        if gate is not None:
            n = n * gate
        if row_gate is not None:
            n = n * row_gate[:, None]
        h1 = res_scale * h + n
    x = None if w_pre is None else h1 * rms_inv(h1, eps) * w_pre
    return (None if y is None else h1), x


def norm_backward(v, g, eps):
    """Gradient of v for the gradient g of N(v)."""
    r = rms_inv(v, eps)
    return r * g - v * r ** 3 * np.mean(g * v, axis=1, keepdims=True)


def block_norm_backward(h1, y=None, *, dh1=None, dx=None, w_post=None, gate=None, row_gate=None,
                        res_scale=1.0, w_pre=None, eps=1e-6):
    """dict of the gradients dh, dy, dw_post, dgate, drow_gate, dw_pre (those that apply)."""
    out = {}
    D = np.zeros_like(h1 if y is None else y) if dh1 is None else dh1.copy()
    if dx is not None:
        D = D + norm_backward(h1, dx * w_pre, eps)
        out["dw_pre"] = np.sum(dx * h1 * rms_inv(h1, eps), axis=0)
    out["dh"] = (res_scale if y is not None else 1.0) * D
    if y is not None:
        n = y if w_post is None else y * rms_inv(y, eps)
        g = 1.0 if gate is None else gate
        rg = 1.0 if row_gate is None else row_gate[:, None]
        w = 1.0 if w_post is None else w_post
        q = D * g * rg * w
        out["dy"] = q if w_post is None else norm_backward(y, q, eps)
        if w_post is not None:
            out["dw_post"] = np.sum(D * rg * g * n, axis=0)
        if gate is not None:
            out["dgate"] = np.sum(D * rg * w * n, axis=0)
        if row_gate is not None:
            out["drow_gate"] = np.sum(D * g * w * n, axis=1)
    return out


def grad_norm(grads):
    return float(np.sqrt(sum(float(np.sum(np.square(g, dtype=np.float64))) for g in grads)))


def clip(grads, max_norm, eps=1e-6):
    """(norm, the clipped tensors)."""
    n = grad_norm(grads)
    c = min(1.0, max_norm / (n + eps))
    return n, [g * c for g in grads]


def adapter_of_position(offsets, NA, T):
    """The adapter of each position, NA for none."""
    a = np.full(T, NA, dtype=np.int64)
    for i in range(NA):
        a[offsets[i]:offsets[i + 1]] = i
    return a


def lora_forward(x, A, B, offsets, y, src_row=None, scale=None):
    """(out, v): v by position (zeros where there is no adapter)."""
    T, NA = x.shape[0], A.shape[0]
    src = np.arange(T) if src_row is None else src_row
    out, v = y.copy(), np.zeros((T, A.shape[1]))
    for a in range(NA):
        p = np.arange(offsets[a], offsets[a + 1])
        v[p] = x[src[p]] @ A[a].T
        out[src[p]] += (1.0 if scale is None else scale[a]) * (v[p] @ B[a].T)
    return out, v


def lora_backward(x, dy, A, B, offsets, v, src_row=None, scale=None, dx=None):
    """(dx_out, dA, dB, u): u by position."""
    T, NA = x.shape[0], A.shape[0]
    src = np.arange(T) if src_row is None else src_row
    dx_out = np.zeros_like(x) if dx is None else dx.copy()
    dA, dB, u = np.zeros(A.shape), np.zeros(B.shape), np.zeros((T, A.shape[1]))
    for a in range(NA):
        p = np.arange(offsets[a], offsets[a + 1])
        s = 1.0 if scale is None else scale[a]
        u[p] = s * (dy[src[p]] @ B[a])
        dx_out[src[p]] += u[p] @ A[a]
        dA[a] = u[p].T @ x[src[p]]
        dB[a] = s * (dy[src[p]].T @ v[p])
    return dx_out, dA, dB, u
