"""Pins of the float64 oracle of the block norms, the clipping and the adapters:
gradients against central differences and torch's float64 autograd, the rest
against closed forms and token-by-token definitions."""
import numpy as np
import pytest
import torch

from oracle import block as ob

EPS = 1e-6


def _args(rng, T, d, post, gate, row_gate, pre):
    return dict(w_post=rng.standard_normal(d) if post else None,
                gate=rng.standard_normal(d) if gate else None,
                row_gate=rng.standard_normal(T) if row_gate else None,
                w_pre=rng.standard_normal(d) if pre else None, res_scale=0.7, eps=EPS)


FLAGS = [(True, True, True, True), (True, False, False, True), (False, True, False, True),
         (True, True, False, False), (False, False, True, False)]


def test_norm_closed_forms():
    v = np.array([[3.0, 4.0], [0.0, 0.0], [1e-3, -1e-3]])
    n = v * ob.rms_inv(v, EPS)
    np.testing.assert_allclose(n[0], v[0] / np.sqrt(12.5 + EPS), rtol=1e-15)
    assert np.all(n[1] == 0.0)
    np.testing.assert_allclose(n[2], [1 / np.sqrt(2), -1 / np.sqrt(2)], rtol=1e-15)
    # pre-norm only leaves no residual; without weights and gates y joins as it is
    h1, x = ob.block_norm_forward(v, w_pre=np.array([2.0, 1.0]))
    assert h1 is None
    np.testing.assert_array_equal(x, n * [2.0, 1.0])
    h1, x = ob.block_norm_forward(v, 2 * v, res_scale=0.5)
    np.testing.assert_allclose(h1, 2.5 * v, rtol=1e-15)
    assert x is None


@pytest.mark.parametrize("post,gate,row_gate,pre", FLAGS)
def test_block_norm_gradients_against_autograd_and_differences(post, gate, row_gate, pre):
    rng = np.random.default_rng(3)
    T, d = 4, 6
    kw = _args(rng, T, d, post, gate, row_gate, pre)
    h, y = rng.standard_normal((T, d)), rng.standard_normal((T, d))
    h1, x = ob.block_norm_forward(h, y, **kw)
    dh1 = rng.standard_normal((T, d))
    dx = rng.standard_normal((T, d)) if pre else None
    g = ob.block_norm_backward(h1, y, dh1=dh1, dx=dx, **kw)

    def loss(h, y, **kw):
        h1, x = ob.block_norm_forward(h, y, **kw)
        return np.sum(h1 * dh1) + (np.sum(x * dx) if pre else 0.0)

    leaves = dict(h=h, y=y, **{n: kw[n] for n in ("w_post", "gate", "row_gate", "w_pre")
                               if kw[n] is not None})
    for name, v in leaves.items():
        num = np.zeros_like(v)
        for i in np.ndindex(v.shape):
            vals = []
            for step in (1e-6, -1e-6):
                w = v.copy()
                w[i] += step
                args = dict(dict(kw, h=h, y=y), **{name: w})
                vals.append(loss(args.pop("h"), args.pop("y"), **args))
            num[i] = (vals[0] - vals[1]) / 2e-6
        np.testing.assert_allclose(g["d" + name], num, rtol=1e-6, atol=1e-7, err_msg=name)

    t = {n: torch.tensor(v, dtype=torch.float64, requires_grad=True) for n, v in leaves.items()}
    unit = lambda v: v / torch.sqrt(v.square().mean(1, keepdim=True) + EPS)
    n = unit(t["y"]) * t["w_post"] if post else t["y"]
    n = n * t.get("gate", 1.0)
    if row_gate:
        n = n * t["row_gate"][:, None]
    o = kw["res_scale"] * t["h"] + n
    total = (o * torch.tensor(dh1)).sum()
    if pre:
        total = total + (unit(o) * t["w_pre"] * torch.tensor(dx)).sum()
    total.backward()
    for name in leaves:
        np.testing.assert_allclose(g["d" + name], t[name].grad.numpy(), rtol=1e-10, atol=1e-12)


def test_combine_and_clip_closed_forms():
    rng = np.random.default_rng(5)
    Y, w = rng.standard_normal((6, 3)), rng.random((2, 3))
    rm = np.array([[5, 0, 3], [1, 2, 4]])
    y = ob.combine(Y, rm, w)
    np.testing.assert_allclose(y[1], w[1, 0] * Y[1] + w[1, 1] * Y[2] + w[1, 2] * Y[4], rtol=1e-15)
    np.testing.assert_allclose(ob.combine(Y, rm, None)[0], Y[5] + Y[0] + Y[3], rtol=1e-15)
    n, out = ob.clip([np.array([3.0, 0.0]), np.array([[4.0]])], 1.0, eps=0.0)
    assert n == 5.0
    np.testing.assert_allclose(out[0], [0.6, 0.0])
    np.testing.assert_allclose(out[1], [[0.8]])
    n, out = ob.clip([np.array([3.0, 4.0])], 6.0)
    np.testing.assert_array_equal(out[0], [3.0, 4.0])


def test_lora_gradients_against_autograd_and_token_by_token():
    rng = np.random.default_rng(7)
    T, K, N, r, NA = 9, 5, 4, 2, 3
    offsets = np.array([0, 4, 4, 7])                    # adapter 1 without rows, two rows without one
    src = rng.permutation(T)
    x, y, A, B = (rng.standard_normal(s) for s in ((T, K), (T, N), (NA, r, K), (NA, N, r)))
    sc, dy, dx = rng.random(NA), rng.standard_normal((T, N)), rng.standard_normal((T, K))
    out, v = ob.lora_forward(x, A, B, offsets, y, src, sc)
    a_of = ob.adapter_of_position(offsets, NA, T)
    for p in range(T):
        t, a = src[p], a_of[p]
        ref = y[t] if a == NA else y[t] + sc[a] * (B[a] @ (A[a] @ x[t]))
        np.testing.assert_allclose(out[t], ref, rtol=1e-13)
    dxo, dA, dB, u = ob.lora_backward(x, dy, A, B, offsets, v, src, sc, dx)
    tx, tA, tB = (torch.tensor(w, requires_grad=True) for w in (x, A, B))
    loss = 0.0
    for p in range(T):
        t, a = int(src[p]), int(a_of[p])
        if a < NA:
            loss = loss + (torch.tensor(dy[t]) * (sc[a] * (tB[a] @ (tA[a] @ tx[t])))).sum()
    loss.backward()
    np.testing.assert_allclose(dxo, dx + tx.grad.numpy(), rtol=1e-12)
    np.testing.assert_allclose(dA, tA.grad.numpy(), rtol=1e-12)
    np.testing.assert_allclose(dB, tB.grad.numpy(), rtol=1e-12)
    assert np.all(dA[1] == 0) and np.all(dB[1] == 0)
