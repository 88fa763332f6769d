"""GPU parity of the global gradient norm and of clipping by it, against float64.

Squares are summed in float64, so the norm is off by its rounding to float32
(2^-24 of it; float64's own error is below 2^-40 of that size for these
lengths); an output adds the factor's rounding, the product's and its store's:
(2^-24 + 2^-24 + u) of the value, u = 2^-8 for bf16 and 0 more for float32."""
import math

import numpy as np
import pytest
import torch

from block_bounds import assert_within
from gpu_util import host, note

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from ragged_grouped_gemm_amd import ops
    ops.moe_version()


def _make(sizes, types, seed=0, scale=1e-3):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * scale * 2.0 ** (i % 9 - 4)).to(DT[t])
            for i, (n, t) in enumerate(zip(sizes, types))]


def _norm64(ts):
    return math.sqrt(math.fsum(float(t.double().square().sum().item()) for t in ts))


def _check(outs, grads, norm, max_norm, eps=1e-6):
    n = _norm64(grads)
    assert abs(float(norm) - n) <= 1.001 * E * n
    c = min(1.0, max_norm / (n + eps))
    for i, (o, g) in enumerate(zip(outs, grads)):
        want = host(g) * c
        u = 2.0 ** -8 if o.dtype == torch.bfloat16 else 0.0
        assert_within(host(o), want, (2.01 * E + u) * np.abs(want), f"out[{i}]")


# one element, lengths around the vector width, the piece and several pieces, empty tensors
SIZES = [[1], [3, 0, 5, 4, 7, 8, 9], [16384], [16383, 16385, 1, 65536 + 3], [200000, 31, 1048577]]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("tin", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("tout", ["f32", "bf16"])
@pytest.mark.parametrize("factor", [0.3, 3.0])
def test_clip_into_new_tensors(sizes, tin, tout, factor):
    from ragged_grouped_gemm_amd import ops
    note(f"clip {sizes} {tin}->{tout} x{factor}")
    types = [tin if tin != "mixed" else ("f32", "bf16")[i % 2] for i in range(len(sizes))]
    gr = _make(sizes, types)
    max_norm = factor * _norm64(gr)
    keep = [t.clone() for t in gr]
    out = [torch.full_like(t, 7.0, dtype=DT[tout]) for t in gr]
    norm = ops.moe_clip_grad_norm(gr, max_norm, out=out)
    _check(out, keep, norm, max_norm)
    assert all(torch.equal(a, b) for a, b in zip(gr, keep))
    assert torch.equal(norm, ops.moe_grad_norm(gr))
    if factor > 1:                      # a factor of one leaves every value as it is
        assert all(torch.equal(o, t.to(o.dtype)) for o, t in zip(out, keep))


@pytest.mark.parametrize("factor", [0.3, 3.0])
def test_clip_in_place(factor):
    from ragged_grouped_gemm_amd import ops
    note(f"clip in place x{factor}")
    gr = _make([5, 70001, 16384, 33], ["f32", "bf16", "bf16", "f32"], 3)
    keep = [t.clone() for t in gr]
    max_norm = factor * _norm64(gr)
    _check(gr, keep, ops.moe_clip_grad_norm(gr, max_norm), max_norm)


@pytest.mark.parametrize("n", [95, 96, 97, 139, 140, 141, 400])
def test_many_tensors_take_several_launches(n):
    """More tensors than one launch holds; a flat buffer's pieces at odd element offsets."""
    from ragged_grouped_gemm_amd import ops
    note(f"clip n={n}")
    rng = np.random.default_rng(n)
    sizes = [int(v) for v in rng.integers(0, 3000, n)]
    gr = _make(sizes, [("f32", "bf16")[int(v)] for v in rng.integers(0, 2, n)], n)
    for dt in (torch.float32, torch.bfloat16):
        flat = torch.full((sum(sizes) + 2,), 5.0, dtype=dt, device="cuda")
        out = list(flat[1:-1].split(sizes))
        max_norm = 0.5 * _norm64(gr)
        _check(out, gr, ops.moe_clip_grad_norm(gr, max_norm, out=out), max_norm)
        assert float(flat[0]) == 5.0 and float(flat[-1]) == 5.0


def test_more_pieces_than_slots():
    """A tensor of more pieces than the workspace has sums, after a batch of small ones."""
    from ragged_grouped_gemm_amd import ops
    note("clip large")
    sizes = [1000] * 96 + [40_000_003]
    gr = _make(sizes, ["f32"] * 97, 1)
    ws = torch.full((ops.moe_grad_norm_workspace_size(97),), 0xA5, dtype=torch.uint8, device="cuda")
    n = _norm64(gr)
    a = ops.moe_grad_norm(gr, ws=ws)
    assert abs(float(a) - n) <= 1.001 * E * n
    assert torch.equal(a, ops.moe_grad_norm(gr, ws=ws))      # same bits, used workspace


def test_extreme_values():
    from ragged_grouped_gemm_amd import ops
    note("clip extreme values")
    f = lambda *v: torch.tensor(v, device="cuda")
    # squares beyond float32's range either way, and zeros
    for v in (3e38, 1e-38, 2.0 ** -140):
        t = [torch.full((1000,), v, device="cuda")]
        want = float(t[0][0]) * math.sqrt(1000.0)
        want = want if want < 3.4028235e38 else math.inf
        got = float(ops.moe_grad_norm(t))
        assert got == want or abs(got - want) <= 1.001 * max(E * want, 2.0 ** -150), (v, got, want)
    z = [torch.zeros(7, device="cuda")]
    assert float(ops.moe_clip_grad_norm(z, 1.0)) == 0.0 and torch.equal(z[0], torch.zeros(7, device="cuda"))
    # an infinite norm scales by zero, a NaN norm makes everything NaN
    a, b = f(1.0, math.inf), f(2.0)
    assert math.isinf(float(ops.moe_clip_grad_norm([a, b], 1.0)))
    assert math.isnan(float(a[1])) and float(a[0]) == 0.0 and float(b) == 0.0
    a, b = f(1.0, math.nan), f(2.0)
    assert math.isnan(float(ops.moe_clip_grad_norm([a, b], 1.0)))
    assert torch.isnan(a).all() and torch.isnan(b).all()
    # max_norm 0 gives zeros, infinity never clips
    a = f(1.0, -2.0)
    ops.moe_clip_grad_norm([a], math.inf)
    assert torch.equal(a, f(1.0, -2.0))
    ops.moe_clip_grad_norm([a], 0.0)
    assert torch.equal(a.abs(), f(0.0, 0.0))


def test_graph_replay_between_eager_calls():
    from ragged_grouped_gemm_amd import ops
    note("clip graph")
    gr = _make([100, 50001, 16384], ["f32", "bf16", "f32"], 4)
    out = [torch.empty_like(t, dtype=torch.float32) for t in gr]
    norm = torch.empty(1, device="cuda")
    ws = torch.empty(ops.moe_grad_norm_workspace_size(3), dtype=torch.uint8, device="cuda")
    max_norm = 0.4 * _norm64(gr)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.moe_clip_grad_norm(gr, max_norm, out=out, norm=norm, ws=ws)
    for seed in range(3):
        for a, b in zip(gr, _make([100, 50001, 16384], ["f32", "bf16", "f32"], 10 + seed)):
            a.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        _check(out, gr, norm, max_norm)
        eager = [torch.empty_like(t) for t in out]
        n2 = ops.moe_clip_grad_norm(gr, max_norm, out=eager)
        assert torch.equal(n2, norm) and all(torch.equal(a, b) for a, b in zip(eager, out))


def test_infinite_max_norm_only_measures():
    """Nothing is scaled, whatever the norm, so long as it is a number."""
    from ragged_grouped_gemm_amd import ops
    note("clip infinite max_norm")
    a = torch.tensor([1.0, math.inf, -3.0], device="cuda")
    out = torch.full_like(a, 7.0)
    assert math.isinf(float(ops.moe_clip_grad_norm([a], math.inf, out=[out])))
    assert torch.equal(out, a)
    assert math.isinf(float(ops.moe_clip_grad_norm([a], math.inf)))
    assert torch.equal(out, a)
    a[0] = math.nan
    assert math.isnan(float(ops.moe_clip_grad_norm([a], math.inf)))
    assert torch.isnan(a).all()


def test_two_streams_at_once():
    """Calls in flight on two streams, each with its own workspace, on inputs made on a third."""
    from ragged_grouped_gemm_amd import ops
    note("clip two streams")
    sizes = [300001, 5, 40000]
    sets = [_make(sizes, ["f32", "bf16", "f32"], 20 + i) for i in range(2)]
    max_norm = [0.4 * _norm64(s) for s in sets]
    want = []
    for s, m in zip(sets, max_norm):
        o = [torch.empty_like(t) for t in s]
        want.append((ops.moe_clip_grad_norm(s, m, out=o), o))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(8):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                o = [torch.empty_like(t) for t in sets[i]]
                got[i].append((ops.moe_clip_grad_norm(sets[i], max_norm[i], out=o), o))
    torch.cuda.synchronize()
    for i in range(2):
        for n, o in got[i]:
            assert torch.equal(n, want[i][0]) and all(torch.equal(a, b) for a, b in zip(o, want[i][1]))
