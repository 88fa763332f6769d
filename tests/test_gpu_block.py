"""The operators together, as a model uses them: blocks of a residual stream (norm, MoE layer,
combine + norm + gate + residual, the next block's norm), adapters beside a shared
projection, and clipping by the norm of every gradient of the step."""
import math

import numpy as np
import pytest
import torch

import synth
from block_bounds import assert_within, norm_fwd_bounds
from gpu_util import host, note, rel_l2
from oracle import block as ob

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from ragged_grouped_gemm_amd import ops
    ops.moe_version()


def _reference(h0, blocks, idx, dh1, dx_last, d):
    """Two blocks in float64 autograd, the experts token by token over the given selection."""
    unit = lambda v: v / torch.sqrt(v.square().mean(1, keepdim=True) + EPS)
    h = h0
    x = unit(h) * blocks[0]["w_pre"]
    for b, sel in zip(blocks, idx):
        w = torch.softmax(b["logits"].gather(1, sel), 1)
        f = b["W1"].shape[1] // 2
        out = torch.zeros_like(h)
        for j in range(sel.shape[1]):
            hid = torch.matmul(b["W1"][sel[:, j]], x[:, :, None])[:, :, 0]
            act = torch.nn.functional.silu(hid[:, :f]) * hid[:, f:]
            out = out + w[:, j:j + 1] * torch.matmul(b["W2"][sel[:, j]], act[:, :, None])[:, :, 0]
        h = 0.75 * h + unit(out) * b["w_post"] * b["gate"]
        x = unit(h) * b["next"]
    return (h * dh1).sum() + (x * dx_last).sum(), h, x


def test_two_blocks_against_autograd():
    """Float32: every gradient of two stacked blocks.  Each library product is held to 1e-5
    of its result elsewhere in these tests; at most 14 of them follow each other here."""
    from ragged_grouped_gemm_amd import ops
    from ragged_grouped_gemm_amd.layer import MoEBlock, MoEFFN
    note("two blocks fp32")
    T, d, f, E, k = 96, 64, 32, 4, 2
    rng = np.random.default_rng(11)
    r = lambda *s: torch.from_numpy(rng.standard_normal(s)).float().cuda()
    w_next = [1 + 0.1 * r(d), 1 + 0.1 * r(d)]
    P = [dict(logits=r(T, E), W1=r(E, 2 * f, d) * d ** -0.5, W2=r(E, d, f) * f ** -0.5,
              w_post=1 + 0.1 * r(d), gate=0.5 * r(d), next=w_next[i]) for i in range(2)]
    P[0]["w_pre"] = 1 + 0.1 * r(d)
    h0, dh1, dx_last = 2 * r(T, d), r(T, d), r(T, d)
    blocks = [MoEBlock(MoEFFN(T, d, f, E, k, dtype=torch.float32, gemm="f32"), res_scale=0.75,
                       eps=EPS) for _ in range(2)]
    W1p = [ops.moe_repack_glu_weights(p["W1"])[0] for p in P]

    def step():
        h, x = h0, None
        for i, (b, p) in enumerate(zip(blocks, P)):
            h, x = b.forward(h, x, p["logits"], W1p[i], p["W2"], w_pre=p.get("w_pre"),
                             w_post=p["w_post"], gate=p["gate"], next_w_pre=p["next"])
        dh, dX = dh1, dx_last
        for i in (1, 0):
            dh, dX = blocks[i].backward(dh, dX, P[i]["logits"], W1p[i], P[i]["W2"])
        assert dX is None
        return h, x, dh

    h, x, dh = step()
    leaves = {n: [p[n].double().requires_grad_(True) for p in P if n in p]
              for n in ("logits", "W1", "W2", "w_post", "gate", "next", "w_pre")}
    hl = h0.double().requires_grad_(True)
    ref = [{n: leaves[n][i] for n in leaves if i < len(leaves[n])} for i in range(2)]
    loss, hr, xr = _reference(hl, ref, [b.ffn.topk_idx.long() for b in blocks], dh1.double(),
                              dx_last.double(), d)
    loss.backward()
    tol = 14e-5
    assert rel_l2(host(h), host(hr)) <= tol and rel_l2(host(x), host(xr)) <= tol
    assert rel_l2(host(dh), host(hl.grad)) <= tol
    for i, b in enumerate(blocks):
        L = b.ffn
        dW1 = ops.moe_repack_glu_weights(L.dW1p, inverse=True)[0]
        got = dict(logits=L.dlogits, W1=dW1, W2=L.dW2, w_post=b.dw_post, gate=b.dgate, next=b.dw_next)
        if i == 0:
            got["w_pre"] = b.dw_pre
        for n, g in got.items():
            assert rel_l2(host(g), host(ref[i][n].grad)) <= tol, (i, n)
    # the same step again gives the same gradients; then all of them clipped as one
    before = [t.clone() for b in blocks for t in b.grads]
    step()
    assert all(torch.equal(a, t) for a, t in zip(before, [t for b in blocks for t in b.grads]))
    norm = blocks[0].clip_grads(1.0, blocks[1].grads)
    n64 = math.sqrt(math.fsum(float(t.double().square().sum()) for t in before))
    assert abs(float(norm) - n64) <= 1.001 * 2.0 ** -24 * n64
    after = math.sqrt(math.fsum(float(t.double().square().sum())
                                for b in blocks for t in b.grads))
    assert abs(after - 1.0) <= 3 * 2.0 ** -24 + 1e-6 / n64


@pytest.mark.parametrize("gemm,gia", [("bf16", False), ("mxfp8", False), ("bf16", True)])
def test_fine_tuning_step_captured(gemm, gia):
    """A bf16 step: block with its own router, a shared projection with adapters of several
    requests, the backward of all, clipping -- eager, and captured and replayed with new
    inputs between eager steps, every replay equal to the eager result."""
    from ragged_grouped_gemm_amd import ops
    from ragged_grouped_gemm_amd.layer import MoEBlock, MoEFFN
    note(f"fine-tuning step {gemm} gate_in_act={gia}")
    T, d, f, E, k, N, rk, NA = 200, 256, 128, 8, 2, 384, 16, 3
    rng = np.random.default_rng(12)
    r = lambda *s: torch.from_numpy(rng.standard_normal(s)).float().cuda()
    bf = lambda t: t.to(torch.bfloat16)
    W1, W2, Wr = bf(r(E, 2 * f, d) * d ** -0.5), bf(r(E, d, f) * f ** -0.5), bf(r(E, d) * d ** -0.5)
    W1p, _ = ops.moe_repack_glu_weights(W1)
    Wl = MoEFFN.mx_weights(W1p, W2, gemm) if gemm != "bf16" else W1p
    Ws = bf(r(1, N, d) * d ** -0.5)
    A, B = bf(r(NA, rk, d) * d ** -0.5), bf(r(NA, N, rk) * rk ** -0.5)
    sc = torch.full((NA,), 0.5, device="cuda")
    w_pre, w_post, gate, w_next = 1 + 0.1 * r(d), 1 + 0.1 * r(d), 0.5 * r(d), 1 + 0.1 * r(d)
    h = bf(2 * r(T, d))
    ids = torch.from_numpy(rng.integers(0, NA + 1, (T, 1)).astype(np.int32)).cuda()
    dy = bf(0.1 * r(T, N))
    off1 = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    kw = dict(w_pre=w_pre, w_post=w_post, gate=gate, next_w_pre=w_next)

    def make():
        L = MoEFFN(T, d, f, E, k, router=True, gemm=gemm, gate_in_act=gia)
        b = MoEBlock(L, res_scale=0.75, eps=EPS)
        z = lambda s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device="cuda")
        f32 = torch.float32
        bufs = dict(y=z((T, N)), v=z((T, rk), f32), dx=z((T, d)), dA=z(A.shape, f32),
                    dB=z(B.shape, f32),
                    ws=z((ops.moe_lora_workspace_size(T, d, N, rk, NA),), torch.uint8),
                    pws=z((ops.moe_permute_workspace_size(T, NA + 1, 1),), torch.uint8),
                    counts=z((NA + 1,), torch.int32), offsets=z((NA + 2,), torch.int32),
                    row_map=z((T, 1), torch.int32), src_row=z((T,), torch.int32))
        return b, bufs

    def step(b, m):
        h1, x = b.forward(h, None, Wr, Wl, W2, **kw)
        ops.moe_permute(None, ids, NA + 1, counts=m["counts"], offsets=m["offsets"],
                        row_map=m["row_map"], src_row=m["src_row"], ws=m["pws"], gather=False)
        ops.moe_grouped_gemm_fwd(x, Ws, off1, y=m["y"])
        plan = dict(src_row=m["src_row"], scale=sc, ws=m["ws"])
        ops.moe_lora_fwd(x, A, B, m["offsets"], m["y"], v_out=m["v"], **plan)
        ops.moe_grouped_gemm_bwd(dy, off1, mode="dgrad", w=Ws, out=m["dx"])
        ops.moe_lora_bwd(x, dy, A, B, m["offsets"], m["v"], dx=m["dx"], dA=m["dA"], dB=m["dB"],
                         **plan)
        dh, _ = b.backward(None, m["dx"], Wr, Wl, W2)
        norm = b.clip_grads(1e-2, (m["dA"], m["dB"]))
        return [h1, x, m["y"], dh, norm, m["dA"], m["dB"], *b.grads]

    b, m = make()
    got = step(b, m)
    torch.cuda.synchronize()
    # the fused combine, norm, gate and residual on the layer's own expert rows
    L = b.ffn
    o = dict(res_scale=0.75, w_post=host(w_post), gate=host(gate), row_gate=None, w_pre=host(w_next))
    w = None if gia else host(L.topk_w)
    y = ob.combine(host(L.Y), host(L.row_map), w)
    yabs = ob.combine(np.abs(host(L.Y)), host(L.row_map), w)
    oh, ox = ob.block_norm_forward(host(h), y, eps=EPS, **o)
    bh, bx = norm_fwd_bounds(host(h), y, yabs, o, EPS, "bf16")
    assert_within(host(got[0]), oh, bh, "h1")
    assert_within(host(got[1]), ox, bx, "x")
    grads = got[5:]
    total = math.sqrt(math.fsum(float(t.double().square().sum()) for t in grads))
    assert abs(total - 1e-2) <= 1e-4 * 1e-2 and float(got[4]) > 1e-2
    assert all(torch.isfinite(t.float()).all() for t in got)

    bg, mg = make()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(bg, mg)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rep = step(bg, mg)
    for i in range(3):
        h.copy_(bf(2 * r(T, d)))
        dy.copy_(bf(0.1 * r(T, N)))
        ids.copy_(torch.from_numpy(rng.integers(0, NA + 1, (T, 1)).astype(np.int32)))
        g.replay()
        torch.cuda.synchronize()
        for a, c in zip(rep, step(b, m)):
            assert torch.equal(a, c), i


def test_block_refuses_what_it_cannot_do():
    from ragged_grouped_gemm_amd.layer import MoEBlock, MoEFFN
    note("block refusals")
    b = MoEBlock(MoEFFN(8, 64, 32, 4, 2))
    t = torch.zeros((8, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    with pytest.raises(ValueError, match="either"):
        b.forward(t, t, None, None, None, w_pre=w)
    with pytest.raises(ValueError, match="either"):
        b.forward(t, None, None, None, None)
    with pytest.raises(RuntimeError, match="before forward"):
        b.backward(t, None, None, None, None)
    with pytest.raises(ValueError, match="empty"):
        b.clip_grads(1.0)
    with pytest.raises(RuntimeError, match="without backward"):
        MoEBlock(MoEFFN(8, 64, 32, 4, 2, backward=False)).backward(t, None, None, None, None)


def test_block_refuses_backward_of_overwritten_state():
    """Inputs that the block's own outputs replace, and a layer that ran again in between."""
    from ragged_grouped_gemm_amd import ops
    from ragged_grouped_gemm_amd.layer import MoEBlock, MoEFFN
    note("block overwritten state")
    T, d, f, E, k = 8, 64, 32, 4, 2
    r = lambda *s: torch.randn(s, device="cuda").bfloat16()
    W1p, _ = ops.moe_repack_glu_weights(r(E, 2 * f, d))
    args = (torch.randn(T, E, device="cuda"), W1p, r(E, d, f))
    w = torch.ones(d, device="cuda")
    L = MoEFFN(T, d, f, E, k)
    a, b = MoEBlock(L), MoEBlock(L)
    h1, x = a.forward(r(T, d), None, *args, w_pre=w, next_w_pre=w)
    with pytest.raises(ValueError, match="write over"):
        a.forward(h1, None, *args, w_pre=w, next_w_pre=w)
    with pytest.raises(ValueError, match="write over"):
        a.forward(h1, x, *args, next_w_pre=w)
    h = r(T, d)
    h2, _ = a.forward(h, None, *args, w_pre=w)
    keep = h2.clone()
    b.forward(h, None, *args, w_pre=w)
    with pytest.raises(RuntimeError, match="another forward"):
        a.backward(r(T, d), None, *args)
    b.backward(r(T, d), None, *args)
    # without a backward, blocks share a layer, and a residual stream stays in one buffer
    L = MoEFFN(T, d, f, E, k, backward=False)
    a = MoEBlock(L)
    h2, _ = a.forward(h, None, *args, w_pre=w)
    assert torch.equal(h2, keep)
    want, _ = MoEBlock(L).forward(keep, None, *args, w_pre=w)
    h3, _ = a.forward(h2, None, *args, w_pre=w)
    assert h3.data_ptr() == h2.data_ptr() and torch.equal(h3, want)
