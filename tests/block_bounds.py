"""Error bounds of the block norms, the clipping and the adapters, element by
element, derived from the arithmetic (none is fitted to a measured error).

u is the store's half step relative to the value (bf16 2^-8, float32 2^-24),
e = 2^-24 one float32 rounding.  Float32 sums over d channels run over at most
32 values per thread, then a tree of 6 and at most 16 waves: at most 54
roundings, 60 with the products; an inverse root of a mean has half the sum's
error and three roundings more (33).  Every quantity is bounded through the
sum of the magnitudes it is made of (the `abs` companions below), so
cancellation costs tolerance where it really occurs."""
import numpy as np

E = 2.0 ** -24
U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _r(v, eps):
    return 1.0 / np.sqrt(np.mean(v * v, axis=1, keepdims=True) + eps)


def _len(v):
    return np.sqrt(np.sum(v * v, axis=1, keepdims=True))


def norm_fwd_bounds(h, y, yabs, kw, eps, dtype):
    """Bounds of (h1, x); yabs: sum_j |w Y| of a combined y, else |y|."""
    u = U[dtype]
    n = a = None
    h1, h1abs = h, np.abs(h)
    if y is not None:
        f = np.ones_like(h)
        for m in (kw["w_post"], kw["gate"]):
            f = f if m is None else f * np.abs(m)
        if kw["row_gate"] is not None:
            f = f * np.abs(kw["row_gate"])[:, None]
        r = _r(y, eps) if kw["w_post"] is not None else 1.0
        n = f * r * yabs
        if kw["w_post"] is not None:
            # an error of the combined y also moves its mean square
            n = n + f * r * np.abs(y) * (_len(yabs) / np.maximum(_len(y), 1e-300))
        sign = np.ones_like(h)
        for m in (kw["w_post"], kw["gate"]):
            sign = sign if m is None else sign * m
        if kw["row_gate"] is not None:
            sign = sign * kw["row_gate"][:, None]
        h1 = kw["res_scale"] * h + sign * r * y
        h1abs = np.abs(kw["res_scale"] * h) + n
    b_h = u * np.abs(h1) + 64 * E * h1abs
    b_x = None
    if kw["w_pre"] is not None:
        r, w = _r(h1, eps), np.abs(kw["w_pre"])
        x = np.abs(h1) * r * w
        b_x = u * x + 64 * E * (x + h1abs * r * w + x * _len(h1abs) / np.maximum(_len(h1), 1e-300))
    return b_h, b_x


def norm_bwd_bounds(h1, y, dh1, dx, kw, eps, dtype, o, rows_added):
    """Bounds of the gradients in o (the oracle's); rows_added: the longest chain of
    float32 additions over tokens."""
    u, b = U[dtype], {}
    Dabs = np.zeros_like(o["dh"]) if dh1 is None else np.abs(dh1)
    if dx is not None:
        r = _r(h1, eps)
        z = np.abs(dx * kw["w_pre"])
        Dabs = Dabs + r * (z + np.abs(h1) * r * r * np.mean(z * np.abs(h1), axis=1, keepdims=True))
        b["dw_pre"] = (64 + rows_added) * E * np.sum(np.abs(dx * h1) * r, axis=0)
    # r^3 (3 x 33), the mean (60) and the products (< 20) inside D
    C = 180
    b["dh"] = u * np.abs(o["dh"]) + C * E * Dabs * (abs(kw["res_scale"]) if y is not None else 1.0)
    if y is not None:
        one = np.ones((1, o["dy"].shape[1]))
        w = one if kw["w_post"] is None else np.abs(kw["w_post"])
        g = one if kw["gate"] is None else np.abs(kw["gate"])
        rg = 1.0 if kw["row_gate"] is None else np.abs(kw["row_gate"])[:, None]
        ry = 1.0 if kw["w_post"] is None else _r(y, eps)
        q, ya = Dabs * w * g, np.abs(y)
        dy = q
        if kw["w_post"] is not None:
            dy = q + ya * ry * ry * np.mean(q * ya, axis=1, keepdims=True)
        b["dy"] = u * np.abs(o["dy"]) + 2 * C * E * ry * rg * dy
        t = Dabs * ya * ry
        if kw["w_post"] is not None:
            b["dw_post"] = (2 * C + rows_added) * E * np.sum(t * rg * g, axis=0)
        if kw["gate"] is not None:
            b["dgate"] = (2 * C + rows_added) * E * np.sum(t * rg * w, axis=0)
        if kw["row_gate"] is not None:
            b["drow_gate"] = 2 * C * E * np.sum(t * g * w, axis=1)
    return b


def assert_within(got, want, bound, what):
    """|got - want| <= bound element by element (equal NaN and infinities pass)."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    with np.errstate(invalid="ignore"):
        bad = ~((np.abs(got - want) <= bound + 2.0 ** -133) | (got == want) |
                (np.isnan(got) & np.isnan(want)))
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        b = np.broadcast_to(bound, want.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside; first at {i}: "
                             f"{got[i]} against {want[i]}, bound {b[i]}")
