"""Cases of the operators around the MoE layer: block norms, gradient clipping, adapters.

``run`` computes each operator either in its plain form (elementary torch
operations in float32, rounded once) or, with ``own`` set, through the
library's entry points.  ``exact`` gives the same results from the
definitions in float64.

Operators (``case["op"]``):

* ``norm_fwd``: h1 = a h + g N(y) w_post, x = N(h1) w_pre, with N(v) = v / sqrt(mean(v^2) + eps),
  g a gate per channel or per token, either stage optional; ``k`` > 0: y is
  first combined from k expert rows per token, y[t] = sum_j w[t, j] Y[row_map[t, j]];
* ``norm_bwd``: its gradients from h1, y, dh1 and dx;
* ``grad_norm``: sqrt of the sum of squares over many tensors;
* ``clip``: the same norm, and every tensor times min(1, max_norm / (norm + 1e-6)), into one buffer;
* ``lora_fwd``: v = x A[a]^T, out = y + s[a] v B[a]^T for each row's adapter a (or none);
* ``lora_bwd``: u = s[a] dy B[a], dx_out = dx + u A[a], dA[a] = u^T x, dB[a] = s[a] dy^T v.
"""
import math

import torch

own = False

EPS = 1e-6
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _norm(name, op, T, d, dtype, post=True, pre=True, gate="channel", k=0):
    c = dict(op=op, T=T, d=d, dtype=dtype, post=post, pre=pre, gate=gate, k=k)
    return dict(c, name=name) if name else c


def _clip(name, op, sizes, dtype="f32", out_dtype="f32", clipped=True):
    """sizes: "rows x cols x count" groups separated by commas (a case holds plain values)."""
    c = dict(op=op, sizes=sizes, dtype=dtype, out_dtype=out_dtype, clipped=clipped)
    return dict(c, name=name) if name else c


def _lora(name, op, T, K, N, r, NA, none=0.1):
    c = dict(op=op, T=T, K=K, N=N, r=r, NA=NA, none=none)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decoding step of eight requests between two blocks: pure latency
        _norm("norm_decode", "norm_fwd", 8, 7168, "bf16"),
        # a training batch of the 7168-wide layer: both norms, channel gate, residual
        _norm("norm_train", "norm_fwd", 16384, 7168, "bf16"),
        # the combine of 4 experts per token closing a 2880-wide layer, with a token gate, ragged batch
        _norm("norm_combine", "norm_fwd", 8191, 2880, "bf16", gate="token", k=4),
        # gradients of the training batch
        _norm("norm_bwd_train", "norm_bwd", 16384, 7168, "bf16"),
        # float32 gradients of a ragged batch, token gate
        _norm("norm_bwd_f32", "norm_bwd", 2049, 2880, "f32", gate="token"),
        # the gradients of many small adapters (two per projection), clipped into new tensors
        _clip("clip_adapters", "clip", "16x2880x61,2880x16x61,1x2880x7"),
        # every gradient of one 32-expert layer, clipped into the bf16 copies that are sent or stored
        _clip("clip_layer", "clip", "184320x2880x1,92160x2880x1,1x184320x1,1x92160x1,32x2880x1",
              out_dtype="bf16"),
        # the norm alone, of bf16 gradients of dense projections
        _clip("norm_of_grads", "grad_norm", "7168x2048x12,2048x7168x12,1x7169x25", dtype="bf16"),
        # one decoding step: 64 requests, 32 resident adapters
        _lora("lora_decode", "lora_fwd", 64, 7168, 7168, 16, 32),
        # a batch of prompts of mixed adapters
        _lora("lora_prompts", "lora_fwd", 8192, 7168, 4096, 32, 16),
        # a short ragged batch at a high rank
        _lora("lora_ragged", "lora_fwd", 1027, 2880, 5760, 64, 5),
        # fine-tuning several adapters at once
        _lora("lora_bwd_train", "lora_bwd", 8192, 4096, 4096, 16, 8),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_fwd", "norm_bwd", "norm_bwd", "clip", "grad_norm", "lora_fwd",
                     "lora_fwd", "lora_bwd"])
    if op in ("norm_fwd", "norm_bwd"):
        d = 8 * _logint(rng, 8, 1024)
        T = min(_logint(rng, 1, 16384), 16384 * 7168 // (2 * d))
        stage = rng.choice(["both", "both", "post", "pre"])
        k = rng.choice([0, 0, 1, 2, 3, 4, 8]) if op == "norm_fwd" and stage != "pre" else 0
        return _norm(None, op, max(1, T // (k + 1)), d, rng.choice(["bf16", "bf16", "f32"]),
                     post=stage != "pre", pre=stage != "post",
                     gate=rng.choice(["none", "channel", "token"]) if stage != "pre" else "none", k=k)
    if op in ("clip", "grad_norm"):
        groups = []
        for _ in range(rng.randint(1, 4)):
            rows, cols = _logint(rng, 1, 4096), _logint(rng, 1, 8192)
            groups.append(f"{rows}x{cols}x{min(_logint(rng, 1, 200), 1 + 60000000 // (rows * cols))}")
        return _clip(None, op, ",".join(groups), rng.choice(["f32", "f32", "bf16"]),
                     rng.choice(["f32", "bf16"]), rng.random() < 0.75)
    T = _logint(rng, 1, 8192)
    K, N = 32 * _logint(rng, 2, 256), 32 * _logint(rng, 2, 256)
    return _lora(None, op, T, K, N, rng.choice([8, 16, 16, 32, 40, 64, 128]), _logint(rng, 1, 48),
                 rng.choice([0.0, 0.1, 0.5]))


# ------------------------------------------------------------------ inputs


def _shapes(case):
    out = []
    for g in case["sizes"].split(","):
        rows, cols, count = (int(v) for v in g.split("x"))
        out += [(rows, cols)] * count
    return out


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def rnd(shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    op = case["op"]
    s = {"case": case}
    if op in ("norm_fwd", "norm_bwd"):
        T, d, k, dt = case["T"], case["d"], case["k"], DT[case["dtype"]]
        stream = 2.0 * (1.0 + 9.0 * (torch.rand(d, generator=g, device="cuda") < 0.01))   # outlier channels
        s["a"] = 0.75 if case["post"] else 1.0
        s["h"] = (torch.randn((T, d), generator=g, device="cuda") * stream).to(dt)
        s["w_pre"] = 1.0 + rnd((d,), 0.1) if case["pre"] else None
        s["y"] = s["w_post"] = s["gate"] = s["row_map"] = s["topk_w"] = None
        if case["post"]:
            s["w_post"] = 1.0 + rnd((d,), 0.1)
            s["gate"] = {"none": None, "channel": rnd((d,), 0.3),
                         "token": torch.sigmoid(rnd((T,)))}[case["gate"]]
            s["y"] = rnd((T * max(k, 1), d), 0.5, dt)
            if k:
                s["row_map"] = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32).view(T, k)
                s["topk_w"] = torch.softmax(rnd((T, k)), dim=1)
        if op == "norm_bwd":
            s["dh1"] = rnd((T, d), 1e-2, dt)
            s["dx"] = rnd((T, d), 1e-2, dt) if case["pre"] else None
    elif op in ("clip", "grad_norm"):
        shapes = _shapes(case)
        dt = DT[case["dtype"]]
        # every tensor at its own scale, as the gradients of different layers are
        sc = [1e-3 * 2.0 ** (i % 7 - 3) for i in range(len(shapes))]
        s["grads"] = [rnd(sh, c, dt) for sh, c in zip(shapes, sc)]
        expect = math.sqrt(sum(sh[0] * sh[1] * c * c for sh, c in zip(shapes, sc)))
        s["max_norm"] = expect * (0.3 if case["clipped"] else 3.0)
        if op == "clip":           # the clipped gradients lie one after another in one buffer
            s["flat"] = torch.empty(sum(t.numel() for t in s["grads"]), dtype=DT[case["out_dtype"]],
                                    device="cuda")
    else:
        T, K, N, r, NA = (case[n] for n in ("T", "K", "N", "r", "NA"))
        bf = torch.bfloat16
        # requests: runs of rows of one adapter (single tokens where there are few rows)
        run = max(1, T // 64)
        ids = torch.randint(0, NA, ((T + run - 1) // run,), generator=g, device="cuda")
        ids = torch.where(torch.rand(ids.shape, generator=g, device="cuda") < case["none"], NA, ids)
        ids = ids.repeat_interleave(run)[:T]
        s["ids"] = ids.to(torch.int32)
        s["A"], s["B"] = rnd((NA, r, K), K ** -0.5, bf), rnd((NA, N, r), 0.5 * r ** -0.5, bf)
        s["scale"] = 0.5 + torch.rand((NA,), generator=g, device="cuda")
        s["x"] = rnd((T, K), 1.0, bf)
        if op == "lora_fwd":
            s["y"] = rnd((T, N), 1.0, bf)
        else:
            s["dy"] = rnd((T, N), 1e-2, bf)
            s["dx"] = rnd((T, K), 1e-2, bf)
        # the batch's plan, shared by all its projections: rows in adapter order
        s["order"] = torch.argsort(ids, stable=True)
        s["counts"] = torch.bincount(ids, minlength=NA + 1).tolist()
        if op == "lora_bwd":       # the low-rank activations that the forward pass kept
            s["v"] = torch.zeros((T, r), device="cuda")
            for a, rows, lo, hi in _segments(s):
                s["v"][lo:hi] = s["x"][rows].float() @ s["A"][a].float().T
    return s


def _views(s, flat):
    """The pieces of a flat buffer that belong to the tensors, in their shapes."""
    return [v.view(t.shape) for v, t in zip(flat.split([t.numel() for t in s["grads"]]), s["grads"])]


def _segments(s):
    """(adapter, its rows, their range in adapter order) for each adapter in use."""
    lo = 0
    for a, n in enumerate(s["counts"][:s["case"]["NA"]]):
        if n:
            yield a, s["order"][lo:lo + n], lo, lo + n
        lo += n


def prepare(case, seed):
    s = _inputs(case, seed)
    if not own:
        return s
    from ragged_grouped_gemm_amd import ops
    op = case["op"]
    if op == "norm_fwd":
        T, d = s["h"].shape
        s["x_out"] = torch.empty_like(s["h"]) if case["pre"] else None
        s["h_out"] = torch.empty_like(s["h"]) if case["post"] else None
    elif op == "norm_bwd":
        T, d = s["h"].shape
        s["ws"] = torch.empty(ops.moe_block_norm_bwd_workspace_size(T, d), dtype=torch.uint8, device="cuda")
    elif op in ("clip", "grad_norm"):
        s["ws"] = torch.empty(ops.moe_grad_norm_workspace_size(len(s["grads"])), dtype=torch.uint8,
                              device="cuda")
        s["norm"] = torch.empty(1, device="cuda")
        if op == "clip":
            s["outs"] = _views(s, s["flat"])
    else:
        T, K, N, r, NA = (case[n] for n in ("T", "K", "N", "r", "NA"))
        _, s["offsets"], _, _, s["src_row"], _ = ops.moe_permute(None, s["ids"].view(T, 1), NA + 1,
                                                                 gather=False)
        s["ws"] = torch.empty(ops.moe_lora_workspace_size(T, K, N, r, NA), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ one pass


def run(state):
    op = state["case"]["op"]
    if own:
        return _own(op, state)
    return {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "clip": _plain_clip,
            "grad_norm": _plain_grad_norm, "lora_fwd": _plain_lora_fwd,
            "lora_bwd": _plain_lora_bwd}[op](state)


def _own(op, s):
    from ragged_grouped_gemm_amd import ops
    if op in ("norm_fwd", "norm_bwd"):
        gate = {"row_gate" if s["case"]["gate"] == "token" else "gate": s["gate"]}
    if op == "norm_fwd":
        h1, x, _ = ops.moe_block_norm_fwd(s["h"], s["y"], w_post=s["w_post"], **gate,
                                          res_scale=s["a"], w_pre=s["w_pre"], eps=EPS,
                                          row_map=s["row_map"], topk_w=s["topk_w"],
                                          h_out=s["h_out"], x_out=s["x_out"])
        return [t for t in (h1, x) if t is not None]
    if op == "norm_bwd":
        g = ops.moe_block_norm_bwd(s["h"], s["y"], dh1=s["dh1"], dx=s["dx"], w_post=s["w_post"],
                                   **gate, res_scale=s["a"], w_pre=s["w_pre"], eps=EPS, ws=s["ws"])
        return [t for t in (g.dh, g.dy, g.dw_post, g.dgate, g.drow_gate, g.dw_pre) if t is not None]
    if op == "grad_norm":
        return ops.moe_grad_norm(s["grads"], norm=s["norm"], ws=s["ws"])
    if op == "clip":
        norm = ops.moe_clip_grad_norm(s["grads"], s["max_norm"], out=s["outs"], norm=s["norm"], ws=s["ws"])
        return [norm, s["flat"]]
    if op == "lora_fwd":
        out, _ = ops.moe_lora_fwd(s["x"], s["A"], s["B"], s["offsets"], s["y"], src_row=s["src_row"],
                                  scale=s["scale"], out=torch.empty_like(s["y"]), ws=s["ws"])
        return out
    dx, dA, dB = ops.moe_lora_bwd(s["x"], s["dy"], s["A"], s["B"], s["offsets"], s["v"],
                                  src_row=s["src_row"], scale=s["scale"], dx=s["dx"],
                                  dx_out=torch.empty_like(s["dx"]), ws=s["ws"])
    return [dx, dA, dB]


def _plain_norm_fwd(s):
    h1 = s["h"].float()
    dt = s["h"].dtype
    res = []
    if s["y"] is not None:
        y = s["y"].float()
        if s["row_map"] is not None:
            T, k = s["row_map"].shape
            y = sum(s["topk_w"][:, j:j + 1] * s["y"][s["row_map"][:, j]].float() for j in range(k))
        n = y * torch.rsqrt(y.square().mean(1, keepdim=True) + EPS) * s["w_post"]
        g = s["gate"]
        if g is not None:
            n = n * (g[:, None] if s["case"]["gate"] == "token" else g)
        h1 = s["a"] * h1 + n
        res.append(h1.to(dt))
    if s["w_pre"] is not None:
        res.append((h1 * torch.rsqrt(h1.square().mean(1, keepdim=True) + EPS) * s["w_pre"]).to(dt))
    return res


def _plain_norm_bwd(s):
    dt = s["h"].dtype
    h1, tot = s["h"].float(), s["dh1"].float()
    dw_pre = None
    if s["dx"] is not None:
        r = torch.rsqrt(h1.square().mean(1, keepdim=True) + EPS)
        dx = s["dx"].float()
        z = dx * s["w_pre"]
        tot = tot + r * (z - h1 * (r * r * (z * h1).mean(1, keepdim=True)))
        dw_pre = (dx * h1 * r).sum(0)
    res = [(s["a"] * tot).to(dt)]
    if s["y"] is not None:
        y, w, gate = s["y"].float(), s["w_post"], s["gate"]
        token = s["case"]["gate"] == "token"
        g = 1.0 if gate is None else gate[:, None] if token else gate
        r = torch.rsqrt(y.square().mean(1, keepdim=True) + EPS)
        q = tot * w * g
        res.append((r * (q - y * (r * r * (q * y).mean(1, keepdim=True)))).to(dt))
        n = tot * y * r
        res.append((n * g).sum(0))
        if gate is not None:
            res.append((n * w).sum(1) if token else (n * w).sum(0))
    return res + ([dw_pre] if dw_pre is not None else [])


def _plain_grad_norm(s):
    return torch.stack([t.float().square().sum(dtype=torch.float64) for t in s["grads"]]).sum() \
        .sqrt().float().view(1)


def _plain_clip(s):
    norm = _plain_grad_norm(s)
    coef = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    for t, o in zip(s["grads"], _views(s, s["flat"])):
        if o.dtype == torch.float32:
            torch.mul(t.float(), coef, out=o)
        else:
            o.copy_(t.float() * coef)
    return [norm, s["flat"]]


def _plain_lora_fwd(s):
    out = s["y"].clone()
    for a, rows, _, _ in _segments(s):
        v = s["x"][rows].float() @ s["A"][a].float().T
        out[rows] = (s["y"][rows].float() + s["scale"][a] * (v @ s["B"][a].float().T)).to(out.dtype)
    return out


def _plain_lora_bwd(s):
    dx = s["dx"].clone()
    dA = torch.zeros(s["A"].shape, device="cuda")
    dB = torch.zeros(s["B"].shape, device="cuda")
    for a, rows, lo, hi in _segments(s):
        dy = s["dy"][rows].float()
        u = s["scale"][a] * (dy @ s["B"][a].float())
        dx[rows] = (s["dx"][rows].float() + u @ s["A"][a].float()).to(dx.dtype)
        dA[a] = u.T @ s["x"][rows].float()
        dB[a] = s["scale"][a] * (dy.T @ s["v"][lo:hi])
    return [dx, dA, dB]


# ------------------------------------------------------------------ least work


def work(case):
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        T, d, k = case["T"], case["d"], case["k"]
        e = 2 if case["dtype"] == "bf16" else 4
        chan = d * 4 * (int(case["pre"]) + int(case["post"]) + int(case["gate"] == "channel"))
        tok = 4 * T * int(case["gate"] == "token") + 8 * T * k
        if op == "norm_fwd":
            n = 1 + (max(k, 1) + 1 if case["post"] else 0) + int(case["pre"])
            fl = (10 + 2 * k) * T * d
        else:
            n = 3 + int(case["pre"]) + (2 if case["post"] else 0)    # h1, dh1, dh; dx; y, dy
            n -= int(not case["pre"])                                 # h1 serves the pre-norm only
            fl, chan, tok = 25 * T * d, 2 * chan, 2 * tok
        return {"bytes": n * T * d * e + chan + tok, "flops": fl}
    if op in ("clip", "grad_norm"):
        n = sum(a * b for a, b in _shapes(case))
        rd = n * (2 if case["dtype"] == "bf16" else 4)
        wr = n * (2 if case["out_dtype"] == "bf16" else 4) if op == "clip" else 0
        return {"bytes": rd + wr, "flops": 2 * n + (n if op == "clip" else 0)}
    T, K, N, r, NA = (case[n] for n in ("T", "K", "N", "r", "NA"))
    used = min(NA, max(1, min(T, 64)))
    w = 2 * used * r * (K + N)
    rows = T * (1.0 - case["none"])
    if op == "lora_fwd":
        return {"bytes": int(2 * rows * K + 4 * T * N + w + 4 * T), "flops": int(2 * rows * r * (K + N))}
    return {"bytes": int(2 * rows * (K + N) + 4 * T * K + 4 * rows * r + w + 4 * NA * r * (K + N)),
            "flops": int(4 * rows * r * (K + N))}


# ------------------------------------------------------------------ float64


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    f64 = lambda t: t.to(torch.float64)
    if op in ("norm_fwd", "norm_bwd"):
        return _exact_norm(case, s, f64)
    if op in ("clip", "grad_norm"):
        total = math.fsum(float(torch.linalg.vector_norm(f64(t)).item()) ** 2 for t in s["grads"])
        norm = torch.tensor([math.sqrt(total)], dtype=torch.float64, device="cuda")
        if op == "grad_norm":
            return norm
        c = min(1.0, s["max_norm"] / (math.sqrt(total) + 1e-6))
        return [norm, torch.cat([f64(t).flatten().mul_(c) for t in s["grads"]])]
    # every row against its own adapter, one adapter's row mask at a time
    out = f64(s["y"] if op == "lora_fwd" else s["dx"]).clone()
    dA = torch.zeros(s["A"].shape, dtype=torch.float64, device="cuda")
    dB = torch.zeros(s["B"].shape, dtype=torch.float64, device="cuda")
    for a in range(case["NA"]):
        t = torch.nonzero(s["ids"] == a).flatten()
        A, B, sc = f64(s["A"][a]), f64(s["B"][a]), f64(s["scale"][a])
        x = f64(s["x"][t])
        if op == "lora_fwd":
            out[t] += sc * torch.mm(torch.mm(x, A.t()), B.t())
        else:
            dy = f64(s["dy"][t])
            v = torch.zeros((s["ids"].numel(), case["r"]), dtype=torch.float64, device="cuda")
            v[s["order"]] = f64(s["v"])
            out[t] += torch.mm(dy, sc * torch.mm(B, A))
            dA[a] = sc * torch.mm(torch.mm(B.t(), dy.t()), x)
            dB[a] = torch.mm(dy.t(), sc * v[t])
    return out if op == "lora_fwd" else [out, dA, dB]


def _exact_norm(case, s, f64):
    def unit(v):
        return v / torch.sqrt(torch.sum(v * v, dim=1, keepdim=True) / v.shape[1] + EPS)

    h = f64(s["h"])
    gate = None if s["gate"] is None else f64(s["gate"])
    shaped = 1.0 if gate is None else gate.view(-1, 1) if case["gate"] == "token" else gate.view(1, -1)
    if case["op"] == "norm_fwd":
        res = []
        if case["post"]:
            y = f64(s["y"])
            if case["k"]:
                y = torch.sum(y[s["row_map"].long()] * f64(s["topk_w"])[:, :, None], dim=1)
            h = s["a"] * h + unit(y) * f64(s["w_post"]) * shaped
            res.append(h)
        if case["pre"]:
            res.append(unit(h) * f64(s["w_pre"]))
        return res
    # gradients by differentiating the float64 forward formulas
    tot = f64(s["dh1"])
    dw_pre = None
    if case["pre"]:
        h.requires_grad_(True)
        w = f64(s["w_pre"]).requires_grad_(True)
        gh, dw_pre = torch.autograd.grad(unit(h) * w, (h, w), grad_outputs=f64(s["dx"]))
        tot = tot + gh
    res = [s["a"] * tot]
    if case["post"]:
        y = f64(s["y"]).requires_grad_(True)
        w = f64(s["w_post"]).requires_grad_(True)
        leaves = [y, w]
        if gate is not None:
            gate = gate.requires_grad_(True)
            shaped = gate.view(-1, 1) if case["gate"] == "token" else gate.view(1, -1)
            leaves.append(gate)
        res += list(torch.autograd.grad(unit(y) * w * shaped, leaves, grad_outputs=tot))
    return res + ([dw_pre] if case["pre"] else [])
