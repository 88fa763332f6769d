"""Tensors of more than 2^31 elements: offsets past 32 bits in the block norms, the clipping
and the adapters.  The rows behind that border are checked against a small call on the
same rows (block norms: bit for bit, a row's result does not depend on its batch) or
against float64."""
import math

import numpy as np
import pytest
import torch

from block_bounds import assert_within
from gpu_util import host, note

pytestmark = [pytest.mark.gpu, pytest.mark.slow]
T, D = 300_001, 7168            # 2.15e9 elements


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from ragged_grouped_gemm_amd import ops
    ops.moe_version()
    yield
    torch.cuda.empty_cache()


def _rows(seed, scale=1.0, width=D):
    """[T, width] bf16, random in the first and last 40 rows, ones between."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = torch.ones((T, width), dtype=torch.bfloat16, device="cuda")
    for part in (t[:40], t[-40:]):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") * scale)
    return t


def test_block_norms_past_32_bits():
    from ragged_grouped_gemm_amd import ops
    note(f"block_norm T={T} d={D}")
    h, y, dx = _rows(1, 2.0), _rows(2), _rows(3, 1e-2)
    w = 1 + 0.1 * torch.randn(D, device="cuda")
    kw = dict(w_post=w, gate=0.5 * w, w_pre=w, res_scale=0.75)
    h1, x, _ = ops.moe_block_norm_fwd(h, y, **kw)
    g = ops.moe_block_norm_bwd(h1, y, dh1=dx, dx=dx, **kw)
    cut = lambda t: torch.cat([t[:40], t[-40:]]).contiguous()
    sh, sx, _ = ops.moe_block_norm_fwd(cut(h), cut(y), **kw)
    sg = ops.moe_block_norm_bwd(cut(h1), cut(y), dh1=cut(dx), dx=cut(dx), **kw)
    for a, b in ((h1, sh), (x, sx), (g.dh, sg.dh), (g.dy, sg.dy)):
        assert torch.equal(cut(a), b)
    assert torch.equal(h1[T // 2], h1[50]) and torch.equal(g.dy[T - 50], g.dy[50])
    # the channel sum over all rows, the equal rows between counted as one
    one = (dx[50].double() * h1[50].double() * torch.rsqrt(h1[50].double().square().mean() + 1e-6))
    want = host(sg.dw_pre) + (T - 80) * host(one)
    assert_within(host(g.dw_pre), want, (1200 + 300) * 2.0 ** -24 * (T * np.abs(host(one)) + 1.0),
                  "dw_pre")


def test_clipping_past_32_bits():
    from ragged_grouped_gemm_amd import ops
    n = 2 ** 31 + 1003
    note(f"clip n={n}")
    a = torch.full((n,), 2.0 ** -10, dtype=torch.bfloat16, device="cuda")
    b = torch.full((5,), 3.0, device="cuda")
    a[-1], a[-2] = 1.5, -2.0
    out = [torch.zeros_like(a), torch.zeros_like(b)]
    total = math.sqrt((n - 2) * 2.0 ** -20 + 1.5 ** 2 + 4.0 + 45.0)
    norm = ops.moe_clip_grad_norm([a, b], 0.5 * total, out=out)
    assert abs(float(norm) - total) <= 1.001 * 2.0 ** -24 * total
    c = 0.5 * total / (total + 1e-6)
    for t, want in ((out[0][-2:], [-2.0 * c, 1.5 * c]), (out[0][:1], [2.0 ** -10 * c]),
                    (out[0][2 ** 31 - 1:2 ** 31 + 1], [2.0 ** -10 * c] * 2), (out[1], [3.0 * c] * 5)):
        want = np.array(want)
        assert_within(host(t), want, (2.0 ** -8 + 2.01 * 2.0 ** -24) * np.abs(want), "out")
    assert int((out[0][2:-2] != out[0][0]).sum()) == 0


def test_adapters_past_32_bits():
    from ragged_grouped_gemm_amd import ops
    K, N, r = D, D, 16
    note(f"lora T={T} K={K} N={N}")
    x, y = _rows(4), _rows(5)
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    A = (torch.randn((2, r, K), generator=g, device="cuda") * K ** -0.5).bfloat16()
    B = (torch.randn((2, N, r), generator=g, device="cuda") * r ** -0.5).bfloat16()
    off = torch.tensor([0, T // 2, T - 3], dtype=torch.int32, device="cuda")
    out, v = ops.moe_lora_fwd(x, A, B, off, y, out=torch.empty_like(y), want_v=True)
    assert torch.equal(out[-3:], y[-3:])
    f = lambda t: host(t).astype(np.float64)
    for a, rows in ((0, slice(0, 40)), (1, slice(T - 40, T - 3))):
        xr, Ar, Br, yr = f(x[rows]), f(A[a]), f(B[a]), f(y[rows])
        vw, mag = xr @ Ar.T, np.abs(xr) @ np.abs(Ar).T
        assert_within(f(v[rows]), vw, 2 * (K / 32 + 40) * 2.0 ** -24 * mag, "v")
        want = yr + vw @ Br.T
        bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -15 + 2.0 ** -13) * (mag @ np.abs(Br).T)
        assert_within(f(out[rows]), want, bound, "out")
    # gradients: dx of the last rows, and the sums over all rows of equal rows between
    dy = torch.zeros_like(y)
    dy[-40:] = 0.5
    dx, dA, dB = ops.moe_lora_bwd(x, dy, A, B, off, v)
    assert not dx[:T - 40].any() and not dA[0].any() and not dB[0].any()
    dyr, xr, vr = f(dy[T - 40:T - 3]), f(x[T - 40:T - 3]), f(v[T - 40:T - 3])
    u = dyr @ f(B[1])
    umag = np.abs(dyr) @ np.abs(f(B[1]))
    t = 2 * (N / 32 + 40) * 2.0 ** -24
    assert_within(f(dA[1]), u.T @ xr, 2 * t * (umag.T @ np.abs(xr)), "dA")
    assert_within(f(dB[1]), dyr.T @ vr, t * (np.abs(dyr).T @ np.abs(vr)), "dB")
    w = u @ f(A[1])
    assert_within(f(dx[T - 40:T - 3]), w, 2.0 ** -8 * np.abs(w) + (2.0 ** -16 + 2 * t) *
                  (umag @ np.abs(f(A[1]))), "dx")
