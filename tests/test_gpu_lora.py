"""GPU parity of the adapters (moe_lora_fwd, moe_lora_bwd) against the float64
oracle, element by element.

Bounds, with e = 2^-24 and u = 2^-8: a matrix-core sum over n bf16 products is
taken in steps of 32 (of 4 in the weight gradients), the waves' and splits'
parts after that, each step within two roundings of the magnitudes added so
far: 2 (n / 32 + 40) e of the sum of magnitudes.  Between the two products the
rank values are split into two bf16 parts, which leaves out at most 2^-16 of
each.  Outputs in bf16 add u of the value."""
import numpy as np
import pytest
import torch

from block_bounds import assert_within
from gpu_util import host, note, rand_bf16
from oracle import block as ob

pytestmark = pytest.mark.gpu
E, U = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from ragged_grouped_gemm_amd import ops
    ops.moe_version()


def _terms(n):
    return 2 * (n / 32 + 40) * E


class Case:
    def __init__(self, T, K, N, r, NA, seed=0, ids=None, scale=True, order=True):
        from ragged_grouped_gemm_amd import ops
        rng = np.random.default_rng([T, K, N, r, NA, seed])
        self.T, self.K, self.N, self.r, self.NA = T, K, N, r, NA
        if ids is None:
            ids = rng.integers(0, NA + 1, T)
        ids = np.asarray(ids if order else np.sort(ids), np.int32)
        self.ids = torch.from_numpy(ids).cuda()
        self.x, self.y = rand_bf16(rng, (T, K)), rand_bf16(rng, (T, N))
        self.A, self.B = rand_bf16(rng, (NA, r, K), K ** -0.5), rand_bf16(rng, (NA, N, r), r ** -0.5)
        self.dy, self.dx = rand_bf16(rng, (T, N), 0.1), rand_bf16(rng, (T, K), 0.1)
        sc = (0.5 + rng.random(NA)).astype(np.float32)
        self.sc = (sc.astype(np.float64), torch.from_numpy(sc).cuda()) if scale else (None, None)
        _, off, _, _, src, _ = ops.moe_permute(None, self.ids.view(T, 1), NA + 1, gather=False)
        self.off = host(off), off
        self.src = (host(src), src) if order else (None, None)
        self.a_of = ob.adapter_of_position(self.off[0], NA, T)

    def forward(self, **kw):
        from ragged_grouped_gemm_amd import ops
        return ops.moe_lora_fwd(self.x[1], self.A[1], self.B[1], self.off[1], self.y[1],
                                src_row=self.src[1], scale=self.sc[1], **kw)

    def check_forward(self, out, v=None):
        want, vw = ob.lora_forward(self.x[0], self.A[0], self.B[0], self.off[0], self.y[0],
                                   self.src[0], self.sc[0])
        zero = np.zeros_like(self.y[0])
        mag, vabs = ob.lora_forward(np.abs(self.x[0]), np.abs(self.A[0]), np.abs(self.B[0]),
                                    self.off[0], zero, self.src[0], self.sc[0])
        bound = U * np.abs(want) + (2.0 ** -16 + _terms(self.K) + _terms(2 * self.r)) * mag \
            + 2 * E * np.abs(want)
        assert_within(host(out), want, np.where(mag > 0, bound, 0.0), "out")
        if v is not None:
            with_a = self.a_of < self.NA
            assert_within(host(v)[with_a], vw[with_a], _terms(self.K) * vabs[with_a], "v")

    def backward(self, v, **kw):
        from ragged_grouped_gemm_amd import ops
        return ops.moe_lora_bwd(self.x[1], self.dy[1], self.A[1], self.B[1], self.off[1], v,
                                src_row=self.src[1], scale=self.sc[1], **kw)

    def check_backward(self, res, v, dx, base=0.0):
        vh = host(v)
        dxh = None if dx is None else host(dx)
        want = ob.lora_backward(self.x[0], self.dy[0], self.A[0], self.B[0], self.off[0], vh,
                                self.src[0], self.sc[0], dxh)
        zero = np.zeros_like(self.x[0])
        mag = ob.lora_backward(np.abs(self.x[0]), np.abs(self.dy[0]), np.abs(self.A[0]),
                               np.abs(self.B[0]), self.off[0], np.abs(vh), self.src[0], self.sc[0],
                               zero)
        rows = int(np.max(np.diff(self.off[0][:self.NA + 1]))) if self.T else 0
        if res[0] is not None:
            b = U * np.abs(want[0]) + (2.0 ** -16 + _terms(self.N) + _terms(2 * self.r)) * mag[0] \
                + 2 * E * np.abs(want[0])
            assert_within(host(res[0]), want[0], np.where(mag[0] > 0, b, 0.0), "dx")
        if res[1] is not None:
            # the waves' rows four at a time, then the parts
            wg = 2 * (rows / 4 + 40) * E
            assert_within(host(res[1]), want[1] + base,
                          (_terms(self.N) + wg) * mag[1] + 2 * E * abs(base), "dA")
            assert_within(host(res[2]), want[2] + base, (wg + 4 * E) * mag[2] + 2 * E * abs(base), "dB")


# (T, K, N, r, NA): single tokens, every rank tile, narrow and odd widths, row tiles of
# both heights with ragged ends, more adapters than rows, many adapters
CASES = [(1, 64, 32, 8, 1), (1, 7168, 7168, 16, 32), (7, 96, 160, 24, 3), (64, 2880, 2880, 16, 32),
         (33, 512, 224, 40, 70), (130, 256, 352, 64, 1), (200, 1024, 96, 128, 2),
         (1027, 320, 2880, 32, 5), (700, 2048, 512, 48, 10), (515, 64, 4096, 80, 3),
         (300, 160, 128, 96, 1), (260, 128, 64, 112, 4), (40, 64, 64, 8, 1022),
         (2048, 512, 512, 16, 1),
         # row tiles of 64; gradients over several chunks of 1024 rows, and one adapter of most rows
         (6200, 96, 160, 16, 2), (9000, 64, 96, 24, 3), (2300, 128, 64, 128, 2),
         # the kernel for many rows at each of its rank steps, columns past whole 64s
         (4200, 288, 256, 16, 3), (4200, 256, 288, 40, 2), (4100, 352, 320, 88, 1),
         (4300, 288, 288, 120, 3)]
# row tiles of 64 in the reduction, at every rank tile count (few columns: the oracle is dense)
MANY = [(17000, 288, 256, 16, 3), (17000, 256, 288, 40, 2), (13300, 352, 320, 88, 1),
        (14700, 288, 288, 120, 3)]      # the kernel for many rows, from 2^22 outputs on
TALL = [(12400, 64, 96, r, 2) for r in (8, 32, 48, 64)] + [(6300, 96, 64, r, 3) for r in (72, 104)]


@pytest.mark.parametrize("T,K,N,r,NA", CASES + TALL + MANY)
def test_forward(T, K, N, r, NA):
    note(f"lora_fwd T={T} K={K} N={N} r={r} NA={NA}")
    c = Case(T, K, N, r, NA)
    y = c.y[1].clone()
    out, v = c.forward(out=torch.full_like(y, 9.0), want_v=True)
    c.check_forward(out, v)
    assert torch.equal(c.y[1], y)
    assert torch.equal(out, c.forward(out=torch.empty_like(y))[0])      # same bits
    inplace, none = c.forward()
    assert none is None and inplace is c.y[1] and torch.equal(inplace, out)


@pytest.mark.parametrize("T,K,N,r,NA", CASES + TALL + MANY)
def test_backward(T, K, N, r, NA):
    note(f"lora_bwd T={T} K={K} N={N} r={r} NA={NA}")
    c = Case(T, K, N, r, NA)
    _, v = c.forward(out=torch.empty_like(c.y[1]), want_v=True)
    res = c.backward(v, dx=c.dx[1], dx_out=torch.empty_like(c.dx[1]))
    c.check_backward(res, v, c.dx[1])
    for a, b in zip(res, c.backward(v, dx=c.dx[1], dx_out=torch.empty_like(c.dx[1]))):
        assert torch.equal(a, b)
    # without the projection's gradient, in place, and each result alone
    new = c.backward(v)
    c.check_backward((new[0], None, None), v, None)
    assert torch.equal(new[1], res[1])
    only = c.backward(v, want_dx=False)
    assert only[0] is None and torch.equal(only[1], res[1]) and torch.equal(only[2], res[2])
    dxi = c.dx[1].clone()
    inp = c.backward(v, dx=dxi, want_dw=False)
    assert inp[0] is dxi and inp[1] is None and torch.equal(dxi, res[0])


@pytest.mark.parametrize("what", ["all none", "all one", "first only", "last only", "alternating"])
@pytest.mark.parametrize("T", [5, 300])
def test_adapter_distributions(what, T):
    note(f"lora ids {what} T={T}")
    NA = 4
    ids = {"all none": np.full(T, NA), "all one": np.full(T, 2),
           "first only": np.where(np.arange(T) == 0, 0, NA),
           "last only": np.where(np.arange(T) == T - 1, 3, NA),
           "alternating": np.arange(T) % 2 * 3}[what]
    c = Case(T, 128, 96, 16, NA, ids=ids)
    out, v = c.forward(out=torch.empty_like(c.y[1]), want_v=True)
    c.check_forward(out, v)
    res = c.backward(v, dx=c.dx[1], dx_out=torch.empty_like(c.dx[1]))
    c.check_backward(res, v, c.dx[1])
    used = set(int(i) for i in ids)
    for a in range(NA):
        if a not in used:
            assert not res[1][a].any() and not res[2][a].any()
    acc = c.backward(v, want_dx=False, dA=torch.full_like(res[1], 0.5),
                     dB=torch.full_like(res[2], 0.5), accumulate=True)
    c.check_backward((None, acc[1], acc[2]), v, c.dx[1], base=0.5)


@pytest.mark.parametrize("T", [50, 400])
def test_rows_in_adapter_order_and_no_scale(T):
    """src_row None: the rows lie in adapter order already, as expert segments do."""
    note(f"lora ordered T={T}")
    c = Case(T, 192, 320, 32, 3, scale=False, order=False)
    out, v = c.forward(out=torch.empty_like(c.y[1]), want_v=True)
    c.check_forward(out, v)
    c.check_backward(c.backward(v, dx=c.dx[1], dx_out=torch.empty_like(c.dx[1])), v, c.dx[1])


def test_rows_without_adapter_keep_every_bit():
    note("lora untouched rows")
    c = Case(90, 64, 64, 8, 2, ids=np.arange(90) % 3)
    y = c.y[1]
    y[2, 0], y[5, 1], y[8, 2] = float("nan"), -0.0, float("inf")
    bits = y.view(torch.int16).clone()
    rows = torch.arange(2, 90, 3)
    out, _ = c.forward(out=torch.full_like(y, 3.0))
    assert torch.equal(out.view(torch.int16)[rows], bits[rows])
    c.forward()
    assert torch.equal(y.view(torch.int16)[rows], bits[rows])


def test_source_rows_outside_the_batch_are_skipped():
    note("lora bad src_row")
    c = Case(40, 64, 64, 8, 2, ids=np.arange(40) % 2)
    ref, _ = c.forward(out=torch.empty_like(c.y[1]))
    src = c.src[1].clone()
    lost = [int(src[3]), int(src[30])]
    src[3], src[30] = -1, 40
    from ragged_grouped_gemm_amd import ops
    out = torch.full_like(c.y[1], 5.0)
    ops.moe_lora_fwd(c.x[1], c.A[1], c.B[1], c.off[1], c.y[1], src_row=src, scale=c.sc[1], out=out)
    keep = [t for t in range(40) if t not in lost]
    assert torch.equal(out[keep], ref[keep])
    assert torch.equal(out[lost], torch.full_like(out[lost], 5.0))


def test_infinite_and_nan_inputs_stay_with_their_row():
    note("lora special values")
    c = Case(64, 128, 128, 16, 3, ids=np.zeros(64))
    ref, _ = c.forward(out=torch.empty_like(c.y[1]))
    c.x[1][5, 3], c.x[1][17, 0] = float("nan"), float("inf")
    out, _ = c.forward(out=torch.empty_like(c.y[1]))
    keep = [t for t in range(64) if t not in (5, 17)]
    assert torch.equal(out[keep], ref[keep])
    assert torch.isnan(out[5]).all()
    # an infinity gives what the formula gives: ranks of zeros make 0 inf = NaN of it, ranks of
    # one sign infinities
    c = Case(3, 64, 64, 8, 1, ids=np.zeros(3))
    c.A[1][:, 1:], c.B[1][:, :, 1:] = 0.0, 0.0
    c.x[1][0], c.x[1][0, 0] = 1.0, float("inf")
    c.A[1][0, 0] = 1.0
    out, v = c.forward(out=torch.empty_like(c.y[1]), want_v=True)
    assert float(v[0, 0]) == float("inf") and torch.isnan(v[0, 1:]).all()
    assert torch.isnan(out[0]).all()
    c.A[1].fill_(1.0)
    b = c.B[1][0, :, 0].clone()
    c.B[1].copy_(b[None, :, None].expand_as(c.B[1]))
    out, v = c.forward(out=torch.empty_like(c.y[1]), want_v=True)
    assert torch.isinf(v[0]).all()
    assert torch.equal(out[0].float(), torch.where(b.float() > 0, float("inf"), -float("inf")))
    _, dA, _ = c.backward(torch.zeros_like(v), want_dx=False)
    assert not torch.isfinite(dA[0, :, 0]).any()
    assert torch.isfinite(dA[0, :, 1:]).all()


def test_graph_replay_with_new_plans():
    """Captured once, replayed with other rows and another grouping, between eager calls."""
    from ragged_grouped_gemm_amd import ops
    note("lora graph")
    T, K, N, r, NA = 300, 512, 256, 16, 6
    c = Case(T, K, N, r, NA)
    ws = torch.empty(ops.moe_lora_workspace_size(T, K, N, r, NA), dtype=torch.uint8, device="cuda")
    out, v = torch.empty_like(c.y[1]), torch.zeros((T, r), device="cuda")
    dxo, dA, dB = torch.empty_like(c.x[1]), torch.empty(c.A[1].shape, device="cuda"), \
        torch.empty(c.B[1].shape, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.forward(out=out, v_out=v, ws=ws)
        c.backward(v, dx=c.dx[1], dx_out=dxo, dA=dA, dB=dB, ws=ws)
    for seed in range(3):
        n = Case(T, K, N, r, NA, seed=seed + 1)
        for a, b in ((c.x, n.x), (c.y, n.y), (c.dy, n.dy), (c.dx, n.dx), (c.off, n.off),
                     (c.src, n.src), (c.A, n.A), (c.B, n.B), (c.sc, n.sc)):
            a[1].copy_(b[1])
        g.replay()
        torch.cuda.synchronize()
        o2, v2 = n.forward(out=torch.empty_like(out), want_v=True)
        n.check_forward(out, v)
        r2 = n.backward(v2, dx=n.dx[1], dx_out=torch.empty_like(dxo))
        for a, b in zip((out, dxo, dA, dB), (o2,) + tuple(r2)):
            assert torch.equal(a, b), seed


def test_empty_batch_gives_zero_weight_gradients():
    from ragged_grouped_gemm_amd import ops
    note("lora T=0")
    bf = torch.bfloat16
    x, y = torch.empty((0, 64), dtype=bf, device="cuda"), torch.empty((0, 32), dtype=bf, device="cuda")
    A = torch.ones((2, 8, 64), dtype=bf, device="cuda")
    B = torch.ones((2, 32, 8), dtype=bf, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    out, v = ops.moe_lora_fwd(x, A, B, off, y, want_v=True)
    assert out.shape == (0, 32) and v.shape == (0, 8)
    dx, dA, dB = ops.moe_lora_bwd(x, y, A, B, off, v, dA=torch.full(A.shape, 3.0, device="cuda"))
    assert dx.shape == (0, 64) and not dA.any() and not dB.any()
    ops.moe_lora_bwd(x, y, A, B, off, v, want_dw=False)


@pytest.mark.parametrize("T,N", [(40, 256), (1500, 1024), (1500, 2816)])
def test_two_streams_at_once(T, N):
    """Calls in flight on two streams that share the adapters and the plan, each with its own
    workspace, give the bits of calls made alone (T = 40 and N = 2816: the kernels for few and
    for many rows)."""
    note(f"lora two streams T={T}")
    c = [Case(T, 256, N, 16, 3, seed=s) for s in (1, 2)]
    for n in ("A", "B", "sc", "off", "src"):
        setattr(c[1], n, getattr(c[0], n))
    def both(k):
        out, v = k.forward(out=torch.empty_like(k.y[1]), want_v=True)
        return [out, v, *k.backward(v, dx=k.dx[1], dx_out=torch.empty_like(k.dx[1]))]
    want = [both(k) for k in c]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(6):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(both(c[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


@pytest.mark.parametrize("T,NA", [(1500, 20), (2600, 40)])
@pytest.mark.parametrize("r", [8, 24, 48, 64, 72, 128])
def test_gradients_of_few_rows_per_adapter_but_one(r, T, NA):
    """Few rows per adapter on average, while one adapter has more than a chunk of them: the
    kernel that gives each wave columns of its own, with and without partial sums, onto zeros
    and onto what is there."""
    note(f"lora skewed rows T={T} r={r}")
    rng = np.random.default_rng([T, r])
    ids = np.where(rng.random(T) < 0.85, 3, rng.integers(0, NA + 1, T))
    c = Case(T, 96, 160, r, NA, ids=ids)
    _, v = c.forward(out=torch.empty_like(c.y[1]), want_v=True)
    c.check_backward(c.backward(v, dx=c.dx[1], dx_out=torch.empty_like(c.dx[1])), v, c.dx[1])
    dA = torch.full(c.A[1].shape, 0.25, device="cuda")
    dB = torch.full(c.B[1].shape, 0.25, device="cuda")
    res = c.backward(v, dA=dA, dB=dB, accumulate=True, want_dx=False)
    c.check_backward(res, v, None, base=0.25)
