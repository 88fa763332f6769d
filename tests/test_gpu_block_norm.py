"""GPU parity of the fused block norms, forward and backward, against the
float64 oracle, element by element within derived bounds (block_bounds)."""
import numpy as np
import pytest
import torch

from block_bounds import assert_within, norm_bwd_bounds, norm_fwd_bounds
from gpu_util import host, note, rand_bf16, rand_f32
from oracle import block as ob

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from ragged_grouped_gemm_amd import ops
    ops.moe_version()


def _vec(rng, n, scale=1.0, mean=0.0):
    v = (mean + scale * rng.standard_normal(n)).astype(np.float32)
    return v.astype(np.float64), torch.from_numpy(v).cuda()


class Case:
    """Inputs of one call: host float64 (`o`) and device (`g`) keyword arguments."""

    def __init__(self, T, d, dtype, flags, seed=0, k=0):
        rng = np.random.default_rng([T, d, seed])
        rand = rand_bf16 if dtype == "bf16" else rand_f32
        self.T, self.d, self.dtype, self.k = T, d, dtype, k
        self.h = rand(rng, (T, d), 2.0)
        self.y = rand(rng, (T * max(k, 1), d), 0.5) if "y" in flags else (None, None)
        self.dh1 = rand(rng, (T, d), 1e-2) if "1" in flags else (None, None)
        self.dx = rand(rng, (T, d), 1e-2) if "x" in flags else (None, None)
        names = {"w_post": ("p", d, 0.2, 1.0), "gate": ("g", d, 0.5, 0.0),
                 "row_gate": ("t", T, 0.5, 0.5), "w_pre": ("x", d, 0.2, 1.0)}
        self.o, self.g = {"res_scale": 0.75}, {"res_scale": 0.75}
        for n, (flag, size, sc, mean) in names.items():
            self.o[n], self.g[n] = _vec(rng, size, sc, mean) if flag in flags else (None, None)
        if k:
            rm = rng.permutation(T * k).astype(np.int32).reshape(T, k)
            self.rm = rm.astype(np.int64), torch.from_numpy(rm).cuda()
            self.w = _vec(rng, (T, k), 0.3, 0.3)

    def combined(self):
        if not self.k:
            return self.y[0], None if self.y[0] is None else np.abs(self.y[0])
        return (ob.combine(self.y[0], self.rm[0], self.w[0]),
                ob.combine(np.abs(self.y[0]), self.rm[0], np.abs(self.w[0])))

    def forward(self, **extra):
        from ragged_grouped_gemm_amd import ops
        if self.k:
            extra = dict(extra, row_map=self.rm[1], topk_w=self.w[1])
        return ops.moe_block_norm_fwd(self.h[1], self.y[1], eps=EPS, **self.g, **extra)

    def check_forward(self, h1, x):
        y, yabs = self.combined()
        oh, ox = ob.block_norm_forward(self.h[0], y, eps=EPS, **self.o)
        bh, bx = norm_fwd_bounds(self.h[0], y, yabs, self.o, EPS, self.dtype)
        if oh is not None:
            assert_within(host(h1), oh, bh, "h1")
        if ox is not None:
            assert_within(host(x), ox, bx, "x")

    def backward(self, **extra):
        from ragged_grouped_gemm_amd import ops
        return ops.moe_block_norm_bwd(self.h[1], self.y[1], dh1=self.dh1[1], dx=self.dx[1], eps=EPS,
                                      **self.g, **extra)

    def check_backward(self, r, base=0.0):
        o = ob.block_norm_backward(self.h[0], self.y[0], dh1=self.dh1[0], dx=self.dx[0], eps=EPS,
                                   **self.o)
        # a row group's share of the rows, the groups 16 apart and the 16 waves
        rows = self.T // 256 + 1 + 40 + 16
        b = norm_bwd_bounds(self.h[0], self.y[0], self.dh1[0], self.dx[0], self.o, EPS, self.dtype,
                            o, rows)
        for n, want in o.items():
            got = host(getattr(r, n))
            if base and n in ("dw_post", "dgate", "dw_pre"):
                want = want + base
                b[n] = b[n] + 2.0 ** -24 * np.abs(want)
            assert_within(got, want, b[n], n)


# widths: one chunk, a wave's row with a partial chunk, each geometry's start and
# end, the widest rows
WIDTHS = [("bf16", 8), ("bf16", 64), ("bf16", 72), ("bf16", 128), ("bf16", 200), ("bf16", 256),
          ("bf16", 264), ("f32", 32), ("f32", 36), ("f32", 100), ("bf16", 504), ("bf16", 512), ("bf16", 520), ("bf16", 1024), ("bf16", 2048),
          ("bf16", 2880), ("bf16", 4104), ("bf16", 7168), ("bf16", 8200), ("bf16", 16384),
          ("bf16", 32768), ("f32", 4), ("f32", 260), ("f32", 1000), ("f32", 2880), ("f32", 7168),
          ("f32", 16384)]
# y, w_post (p), gate (g), row gate (t), w_pre and dx (x), dh1 (1)
FLAGS = ["ypgx1", "yptx1", "ypgtx", "yp1", "ygt1", "yx1", "y1", "x1", "x"]


@pytest.mark.parametrize("dtype,d", WIDTHS)
def test_forward_widths(dtype, d):
    note(f"block_norm_fwd {dtype} d={d}")
    c = Case(13, d, dtype, "ypgtx")
    h1, x, _ = c.forward()
    c.check_forward(h1, x)


@pytest.mark.parametrize("dtype,d", WIDTHS)
def test_backward_widths(dtype, d):
    note(f"block_norm_bwd {dtype} d={d}")
    c = Case(13, d, dtype, "ypgtx1")
    c.check_backward(c.backward())


@pytest.mark.parametrize("flags", FLAGS)
@pytest.mark.parametrize("dtype,T,d", [("bf16", 1, 2880), ("bf16", 131, 512), ("f32", 67, 1032),
                                       ("bf16", 77, 40), ("f32", 39, 60), ("bf16", 45, 248)])
def test_every_combination_of_stages(dtype, T, d, flags):
    note(f"block_norm {dtype} T={T} d={d} {flags}")
    c = Case(T, d, dtype, flags)
    h1, x, _ = c.forward()
    assert (h1 is None) == ("y" not in flags) and (x is None) == ("x" not in flags)
    c.check_forward(h1, x)
    c.check_backward(c.backward())


@pytest.mark.parametrize("T", [1, 511, 512, 513, 2500, 40000])
@pytest.mark.parametrize("dtype,d", [("bf16", 256), ("bf16", 2048), ("f32", 1024), ("bf16", 56),
                                     ("f32", 16)])
def test_many_rows(dtype, d, T):
    """Row counts around the backward's row groups; the same call twice gives the same bits."""
    note(f"block_norm rows {dtype} T={T} d={d}")
    c = Case(T, d, dtype, "ypgtx1")
    h1, x, _ = c.forward()
    c.check_forward(h1, x)
    r = c.backward()
    c.check_backward(r)
    for a, b in zip(r, c.backward()):
        assert torch.equal(a, b)


@pytest.mark.parametrize("k", [1, 2, 3, 4, 6, 8, 32])
@pytest.mark.parametrize("dtype,T,d", [("bf16", 37, 2880), ("f32", 50, 128), ("bf16", 9, 7168),
                                       ("bf16", 33, 64)])
def test_combine_fused(dtype, T, d, k):
    """y combined from expert rows; the kept y is the combine's own result."""
    from ragged_grouped_gemm_amd import ops
    note(f"block_norm combine {dtype} T={T} d={d} k={k}")
    c = Case(T, d, dtype, "ypgtx", k=k)
    h1, x, y = c.forward(want_y=True)
    c.check_forward(h1, x)
    assert torch.equal(y, ops.moe_unpermute_combine(c.y[1], c.rm[1], c.w[1]))
    assert c.forward()[2] is None
    # unit weights, and row ids outside the rows (row 0 is read, as the combine does)
    bad = c.rm[1].clone()
    bad[0, 0], bad[T - 1, k - 1] = -3, T * k
    got = ops.moe_block_norm_fwd(c.h[1], c.y[1], eps=EPS, row_map=bad, want_y=True, **c.g)[2]
    assert torch.equal(got, ops.moe_unpermute_combine(c.y[1], bad, None))


def test_empty_batch_gives_zero_channel_gradients():
    from ragged_grouped_gemm_amd import ops
    note("block_norm T=0")
    d = 64
    e = torch.empty((0, d), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(d, device="cuda")
    h1, x, _ = ops.moe_block_norm_fwd(e, e, w_post=w, gate=w, w_pre=w)
    assert h1.shape == x.shape == (0, d)
    r = ops.moe_block_norm_bwd(e, e, dh1=e, dx=e, w_post=w, gate=w, w_pre=w,
                               dw_pre=torch.full((d,), 3.0, device="cuda"))
    for g in (r.dw_post, r.dgate, r.dw_pre):
        assert torch.equal(g, torch.zeros(d, device="cuda"))
    r = ops.moe_block_norm_bwd(e, e, dh1=e, dx=e, w_post=w, gate=w, w_pre=w, accumulate=True,
                               dw_pre=torch.full((d,), 3.0, device="cuda"), dw_post=w.clone(),
                               dgate=w.clone())
    assert torch.equal(r.dw_pre, torch.full((d,), 3.0, device="cuda")) and torch.equal(r.dgate, w)


def test_accumulate_and_wanted_outputs_only():
    note("block_norm accumulate")
    c = Case(600, 520, "bf16", "ypgx1")
    ones = lambda: torch.full((520,), 2.0, device="cuda")
    r = c.backward(accumulate=True, dw_post=ones(), dgate=ones(), dw_pre=ones())
    c.check_backward(r, base=2.0)


@pytest.mark.parametrize("dtype,d", [("bf16", 512), ("bf16", 2880), ("f32", 2880)])
def test_outputs_in_the_inputs_memory(dtype, d):
    """Each output may be one of the row's own inputs: bit for bit as with separate tensors."""
    note(f"block_norm in place {dtype} d={d}")
    c = Case(300, d, dtype, "ypgtx1")
    h1, x, _ = c.forward()
    g = c.backward()
    a = Case(300, d, dtype, "ypgtx1")
    ah, ax, _ = a.forward(h_out=a.h[1], x_out=a.y[1])
    assert ah is a.h[1] and torch.equal(ah, h1) and torch.equal(ax, x)
    a = Case(300, d, dtype, "ypgtx1")
    r = a.backward(dh=a.dh1[1], dy=a.y[1])
    for p, q in zip(r, g):
        assert torch.equal(p, q)
    a = Case(300, d, dtype, "ypgtx1")
    r = a.backward(dh=a.h[1], dy=a.dx[1])
    for p, q in zip(r, g):
        assert torch.equal(p, q)


def test_zero_rows_infinities_and_nan_stay_in_their_rows():
    """A row of zeros norms to zeros; NaN and infinities reach their own row only."""
    note("block_norm special values")
    T, d = 40, 2880
    c = Case(T, d, "bf16", "ypgx1")
    ref_h, ref_x, _ = c.forward()
    ref = c.backward()
    c.y[1][3] = 0.0
    c.h[1][3] = 0.0
    c.y[1][7, 11] = float("nan")
    c.y[1][9, 0] = float("inf")
    h1, x, _ = c.forward()
    assert torch.equal(h1[3], torch.zeros_like(h1[3])) and torch.equal(x[3], h1[3])
    assert torch.isnan(x[7]).all() and torch.isnan(h1[9, 0])
    keep = [t for t in range(T) if t not in (3, 7, 9)]
    assert torch.equal(h1[keep], ref_h[keep]) and torch.equal(x[keep], ref_x[keep])
    r = c.backward()
    assert torch.equal(r.dh[keep], ref.dh[keep]) and torch.equal(r.dy[keep], ref.dy[keep])
    assert torch.isfinite(r.dh).all()
    assert torch.isnan(r.dy[7]).all()
    assert torch.isnan(r.dw_post[11])


def test_gradients_against_differences():
    """The backward against central differences of the float32 forward: a change of one
    input by s moves the loss by s times its gradient, to the curvature of the
    norm (s^2 with |h| ~ 1) and the forward's float32 rounding (64 e of the terms, over s)."""
    from ragged_grouped_gemm_amd import ops
    note("block_norm differences")
    c = Case(3, 64, "f32", "ypgtx1")
    h1, x, _ = c.forward()
    r = ops.moe_block_norm_bwd(h1, c.y[1], dh1=c.dh1[1], dx=c.dx[1], eps=EPS, **c.g)

    def loss(**ch):
        a = dict(dict(c.g, h=c.h[1], y=c.y[1]), **ch)
        o, xx, _ = ops.moe_block_norm_fwd(a.pop("h"), a.pop("y"), eps=EPS, **a)
        terms = torch.cat([(o.double() * c.dh1[1]).flatten(), (xx.double() * c.dx[1]).flatten()])
        return terms.sum().item(), terms.abs().sum().item()

    s = 2.0 ** -7
    for name in ("h", "y", "w_post", "gate", "row_gate", "w_pre"):
        src = {"h": c.h[1], "y": c.y[1]}.get(name, c.g.get(name))
        grad = getattr(r, "d" + name)
        for i in ((0,), (src.numel() // 2,), (src.numel() - 1,)):
            v = []
            for sign in (1.0, -1.0):
                t = src.clone()
                t.view(-1)[i] += sign * s
                v.append(loss(**{name: t}))
            num, size = (v[0][0] - v[1][0]) / (2 * s), v[0][1]
            tol = 64 * 2.0 ** -24 * size / s + 16 * s * s * float(grad.abs().max())
            assert abs(num - float(grad.view(-1)[i])) <= tol, (name, i, num, float(grad.view(-1)[i]))


def test_other_stream_and_graph_replay():
    """On a side stream, and captured in a graph that is replayed with new inputs between
    eager calls and synchronizations: every replay equals the eager result."""
    from ragged_grouped_gemm_amd import ops
    note("block_norm graph")
    c = Case(700, 2880, "bf16", "ypgtx1", k=0)
    T, d = c.h[1].shape
    ws = torch.empty(ops.moe_block_norm_bwd_workspace_size(T, d), dtype=torch.uint8, device="cuda")
    new = lambda: torch.empty_like(c.h[1])
    bufs = dict(h_out=new(), x_out=new())
    gb = dict(dh=new(), dy=new(), dw_post=torch.empty(d, device="cuda"),
              dgate=torch.empty(d, device="cuda"), dw_pre=torch.empty(d, device="cuda"),
              drow_gate=torch.empty(T, device="cuda"), ws=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = c.forward()[:2] + tuple(c.backward())
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(side, c.forward()[:2] + tuple(c.backward())):
        assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.forward(**bufs)
        c.backward(**gb)
    for seed in range(3):
        n = Case(700, 2880, "bf16", "ypgtx1", seed=seed + 5)
        for a, b in ((c.h, n.h), (c.y, n.y), (c.dh1, n.dh1), (c.dx, n.dx)):
            a[1].copy_(b[1])
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (bufs["h_out"], bufs["x_out"], gb["dh"], gb["dy"], gb["dw_post"],
                                   gb["dgate"], gb["drow_gate"], gb["dw_pre"])]
        for a, b in zip(got, c.forward()[:2] + tuple(c.backward())):
            assert torch.equal(a, b), seed


@pytest.mark.parametrize("flags", ["ypgx1", "yptx1", "ypgtx", "ygt1", "y1", "yx1", "x"])
@pytest.mark.parametrize("dtype,T,d", [("bf16", 600, 8200), ("f32", 530, 4100), ("bf16", 300, 20480),
                                       ("f32", 300, 8256)])
def test_wide_rows_share_blocks(dtype, T, d, flags):
    """More rows than blocks, where a thread holds two chunks of a row or four."""
    note(f"block_norm wide {dtype} T={T} d={d} {flags}")
    c = Case(T, d, dtype, flags)
    h1, x, _ = c.forward()
    c.check_forward(h1, x)
    r = c.backward()
    c.check_backward(r)
    for a, b in zip(r, c.backward()):
        assert a is b is None or torch.equal(a, b)
