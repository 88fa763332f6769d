"""Host-side checks of the block norms, the clipping and the adapters (no GPU):
struct layouts, refused arguments, workspace sizes."""
import ctypes
import math
import os
import shutil
import subprocess

import pytest
import torch

from ragged_grouped_gemm_amd import _lib, ops

INV, UNS, WSP = _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED, _lib.MOE_ERR_WORKSPACE
F32, BF16 = _lib.MOE_F32, _lib.MOE_BF16


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def P(i):
    """Distinct 16-byte aligned addresses 16 MiB apart, never dereferenced."""
    return (i + 1) << 24


def _make(cls, **kw):
    a = cls(ctypes.sizeof(cls))
    for n, v in kw.items():
        setattr(a, n, v)
    return a


def _status(fn, a, **kw):
    b = type(a)()
    ctypes.pointer(b)[0] = a
    for n, v in kw.items():
        setattr(b, n, v)
    return fn(ctypes.byref(b), None)


def test_struct_layouts_match_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = {"moe_block_norm_fwd_args_t": _lib.BlockNormFwdArgs,
               "moe_block_norm_bwd_args_t": _lib.BlockNormBwdArgs, "moe_tensor_t": _lib.TensorT,
               "moe_lora_fwd_args_t": _lib.LoraFwdArgs, "moe_lora_bwd_args_t": _lib.LoraBwdArgs}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "moe.h"', "int main(void){"]
    for cname, py in structs.items():
        lines.append(f'printf("{cname} size %zu\\n", sizeof({cname}));')
        lines += [f'printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));' for f, _ in py._fields_]
    src, exe = tmp_path / "probe.c", tmp_path / "probe"
    src.write_text("\n".join(lines + ["return 0;}"]))
    subprocess.run([cc, "-I", os.path.dirname(_lib.HEADER), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    got = {tuple(l.split()[:2]): int(l.split()[2]) for l in out.splitlines()}
    for cname, py in structs.items():
        assert got[(cname, "size")] == ctypes.sizeof(py), cname
        for f, _ in py._fields_:
            assert got[(cname, f)] == getattr(py, f).offset, (cname, f)


def test_block_norm_fwd_refusals(lib):
    fn = lib.moe_block_norm_fwd
    a = _make(_lib.BlockNormFwdArgs, dtype=BF16, T=4, d=64, res_scale=1.0, eps=1e-6, h=P(0), y=P(1),
              w_post=P(2), gate=P(3), row_gate=P(4), w_pre=P(5), h_out=P(6), x_out=P(7))
    assert fn(None, None) == INV
    for bad in (dict(struct_size=8), dict(T=-1), dict(d=0), dict(d=60), dict(dtype=7), dict(eps=0.0),
                dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(res_scale=math.nan),
                dict(h=None), dict(h_out=None), dict(x_out=None), dict(w_pre=None),
                dict(h=P(0) + 2), dict(y=P(1) + 8), dict(w_post=P(2) + 4), dict(x_out=P(7) + 8),
                dict(y_out=P(8)), dict(topk_w=P(8)),                       # without row_map
                dict(row_map=P(8), k=0), dict(row_map=P(8), k=33),
                dict(row_map=P(8), k=1 << 30),
                dict(h_out=P(0) + 128), dict(x_out=P(6)), dict(x_out=P(6) + 16),
                dict(h_out=P(1) + 16), dict(row_map=P(8), k=2, h_out=P(1)),
                dict(row_map=P(8), k=2, h_out=P(1) + 512),
                dict(row_map=P(8), k=2, y_out=P(0))):
        assert _status(fn, a, **bad) == INV, bad
    # only the next norm: nothing of the block's output may be given
    pre = dict(y=None, w_post=None, gate=None, row_gate=None, h_out=None)
    for n in pre:
        assert _status(fn, a, **{k: v for k, v in pre.items() if k != n}) == INV, n
    assert _status(fn, a, **pre, w_pre=None, x_out=None) == INV
    assert _status(fn, a, d=32776) == UNS and _status(fn, a, dtype=F32, d=16388) == UNS
    assert _status(fn, a, T=0) == 0
    assert _status(fn, a, **pre, T=0) == 0


def test_block_norm_bwd_refusals(lib):
    fn = lib.moe_block_norm_bwd
    need = lib.moe_block_norm_bwd_workspace_size(4, 64)
    assert need >= 2 * 64 * 4 and lib.moe_block_norm_bwd_workspace_size(0, 64) == 0
    a = _make(_lib.BlockNormBwdArgs, dtype=BF16, T=4, d=64, res_scale=1.0, eps=1e-6, h1=P(0), y=P(1),
              dh1=P(2), dx=P(3), w_post=P(4), gate=P(5), row_gate=P(6), w_pre=P(7), dh=P(8), dy=P(9),
              dw_post=P(10), dgate=P(11), drow_gate=P(12), dw_pre=P(13), ws=P(14), ws_bytes=need)
    assert fn(None, None) == INV
    for bad in (dict(struct_size=16), dict(T=-1), dict(d=0), dict(d=4), dict(dtype=2),
                dict(eps=0.0), dict(res_scale=math.inf), dict(dx=None), dict(w_pre=None),
                dict(h1=None), dict(dy=None), dict(dh=None), dict(w_post=None), dict(gate=None),
                dict(row_gate=None), dict(h1=P(0) + 2), dict(dy=P(9) + 8), dict(ws=P(14) + 4),
                dict(dh=P(2) + 128), dict(dy=P(8)), dict(dy=P(8) + 64), dict(dh=P(1) + 16),
                dict(ws=P(8) - need + 16), dict(ws=P(0)), dict(ws=P(13))):
        assert _status(fn, a, **bad) == INV, bad
    # neither stage; a lone output stage without a gradient to pass on
    assert _status(fn, a, y=None, w_post=None, gate=None, row_gate=None, dy=None, dw_post=None,
                   dgate=None, drow_gate=None, dx=None, w_pre=None, dw_pre=None) == INV
    assert _status(fn, a, dx=None, w_pre=None, dw_pre=None, dh1=None) == INV
    assert _status(fn, a, ws_bytes=need - 1) == WSP and _status(fn, a, ws=None) == WSP
    assert _status(fn, a, d=32776) == UNS


def test_clip_refusals(lib):
    T = _lib.TensorT
    nb = lib.moe_grad_norm_workspace_size(2)
    inf, norm, ws = math.inf, P(8), P(9)

    def clip(ts, max_norm=1.0, eps=1e-6, norm=norm, ws=ws, nb=nb, n=None):
        arr = (T * max(len(ts), 1))(*ts)
        return lib.moe_clip_grad_norm(arr, len(ts) if n is None else n, max_norm, eps, norm, ws, nb,
                                      None)

    good = [T(P(0), P(1), 100, F32, BF16), T(P(2), P(2), 100, BF16, BF16)]
    for kw in (dict(max_norm=-1.0), dict(max_norm=math.nan), dict(eps=0.0), dict(eps=math.nan),
               dict(eps=inf), dict(norm=None), dict(ws=None), dict(ws=P(9) + 8), dict(n=-1),
               dict(norm=P(1) + 16), dict(norm=P(9)), dict(ws=P(1) - 16), dict(ws=P(0))):
        assert clip(good, **kw) == INV, kw
    assert clip(good, nb=nb - 1) == WSP
    assert lib.moe_clip_grad_norm(None, 2, 1.0, 1e-6, norm, ws, nb, None) == INV
    assert lib.moe_grad_norm(None, 2, norm, ws, nb, None) == INV
    for bad in (T(None, P(3), 4, F32, F32), T(P(3), None, 4, F32, F32), T(P(3), P(4), -1, F32, F32),
                T(P(3) + 2, P(4), 4, F32, F32), T(P(3), P(4) + 1, 4, F32, BF16),
                T(P(3), P(4), 4, 5, F32), T(P(3), P(4), 4, F32, 5), T(P(3), P(4), 1 << 43, F32, F32),
                T(P(3), P(3), 4, F32, BF16),              # in place, of another type
                T(P(3), P(3) + 4, 4, F32, F32),           # over itself, shifted
                T(P(3), P(1) + 198, 4, F32, BF16),        # the end of the first output
                T(P(3), P(0) + 396, 4, F32, F32),         # the end of the first input
                T(P(2), P(2), 100, BF16, BF16),           # the second tensor again
                T(P(2), P(4), 100, BF16, BF16),           # reads what another clips in place
                T(P(1) + 100, P(4), 4, F32, F32)):        # reads the first output
        assert clip(good + [bad]) == INV, (bad.data, bad.out)
    one = (T * 1)(T(P(0), None, 4, 9, 0))
    assert lib.moe_grad_norm(one, 1, norm, ws, nb, None) == INV


def _lora(cls, nb, **kw):
    a = dict(dtype=BF16, T=8, K=64, N=96, r=16, NA=3, x=P(0), A=P(1), B=P(2), scale=P(3),
             offsets=P(4), src_row=P(5), ws=P(6), ws_bytes=nb)
    a.update(kw)
    return _make(cls, **a)


SIZE_REFUSALS = (dict(struct_size=8), dict(T=-1), dict(K=0), dict(K=48), dict(N=40), dict(r=0),
                 dict(r=12), dict(T=(1 << 30) + 1), dict(K=1 << 21), dict(N=1 << 21), dict(NA=0), dict(NA=1024), dict(dtype=9))


def test_lora_refusals(lib):
    nb = lib.moe_lora_workspace_size(8, 64, 96, 16, 3)
    fwd = _lora(_lib.LoraFwdArgs, nb, y=P(7), out=P(8), v_out=P(9))
    fn = lib.moe_lora_fwd
    assert fn(None, None) == INV
    for bad in SIZE_REFUSALS + (dict(x=None), dict(A=None), dict(B=None), dict(y=None),
                                dict(out=None), dict(offsets=None), dict(x=P(0) + 2),
                                dict(v_out=P(9) + 4), dict(out=P(7) + 64), dict(out=P(0) + 64),
                                dict(out=P(1)), dict(out=P(6)), dict(v_out=P(8)), dict(v_out=P(0)),
                                dict(v_out=P(6)), dict(ws=P(7))):
        assert _status(fn, fwd, **bad) == INV, bad
    assert _status(fn, fwd, dtype=F32) == UNS and _status(fn, fwd, r=136) == UNS
    assert _status(fn, fwd, ws=None) == WSP and _status(fn, fwd, ws_bytes=nb - 1) == WSP
    assert _status(fn, fwd, T=0) == 0

    bwd = _lora(_lib.LoraBwdArgs, nb, dy=P(7), v=P(8), dx=P(9), dx_out=P(10), dA=P(11), dB=P(12))
    fn = lib.moe_lora_bwd
    assert fn(None, None) == INV
    for bad in SIZE_REFUSALS + (dict(x=None), dict(dy=None), dict(A=None), dict(B=None), dict(v=None),
                                dict(offsets=None), dict(dx_out=None, dx=None, dA=None, dB=None),
                                dict(dx_out=None),                    # dx without a place for the sum
                                dict(dx_out=P(9) + 64), dict(dx_out=P(0)), dict(dx_out=P(7)),
                                dict(dA=P(11) + 4), dict(dA=P(0)), dict(dB=P(11)), dict(dA=P(10)),
                                dict(ws=P(12))):
        assert _status(fn, bwd, **bad) == INV, bad
    assert _status(fn, bwd, dtype=F32) == UNS and _status(fn, bwd, r=256) == UNS
    assert _status(fn, bwd, ws=None) == WSP and _status(fn, bwd, ws_bytes=nb - 1) == WSP


def test_binding_refuses_host_tensors_and_wrong_shapes():
    """Errors of the binding itself, before the library is called."""
    h, w = torch.zeros(4, 64), torch.ones(64)
    with pytest.raises(ValueError, match="GPU"):
        ops.moe_block_norm_fwd(h, w_pre=w)
    with pytest.raises(ValueError, match="GPU"):
        ops.moe_block_norm_bwd(h, dx=h, w_pre=w)
    with pytest.raises(ValueError, match="GPU"):
        ops.moe_grad_norm([h])
    with pytest.raises(ValueError, match="GPU"):
        ops.moe_clip_grad_norm([h], 1.0)
    with pytest.raises(ValueError, match="w_pre"):
        ops.moe_block_norm_fwd(h, w_pre=torch.ones(60))
    with pytest.raises(TypeError, match="w_pre"):
        ops.moe_block_norm_fwd(h, w_pre=w.double())
    with pytest.raises(ValueError, match="y must be"):
        ops.moe_block_norm_fwd(h, torch.zeros(8, 64))
    with pytest.raises(ValueError, match="contiguous"):
        ops.moe_block_norm_fwd(torch.zeros(64, 4).t(), w_pre=w)
    with pytest.raises(TypeError):
        ops.moe_block_norm_fwd(h.half(), w_pre=w)
    with pytest.raises(ValueError, match="row_map"):
        ops.moe_block_norm_fwd(h, h, want_y=True)
    with pytest.raises(ValueError, match="accumulate"):
        ops.moe_block_norm_bwd(h, dx=h, w_pre=w, accumulate=True)
    with pytest.raises(ValueError, match="empty"):
        ops.moe_grad_norm([])
    with pytest.raises(ValueError, match="outputs"):
        ops.moe_clip_grad_norm([h], 1.0, out=[])
    with pytest.raises(ValueError, match="out"):
        ops.moe_clip_grad_norm([h], 1.0, out=[w])
    bf = torch.bfloat16
    x, A, B = torch.zeros(4, 64, dtype=bf), torch.zeros(2, 8, 64, dtype=bf), torch.zeros(2, 32, 8, dtype=bf)
    y, off = torch.zeros(4, 32, dtype=bf), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        ops.moe_lora_fwd(x, A, B, off, y)
    with pytest.raises(ValueError, match="offsets"):
        ops.moe_lora_fwd(x, A, B, off[:2], y)
    with pytest.raises(ValueError, match="A must be"):
        ops.moe_lora_fwd(x, A[:, :, :32].contiguous(), B, off, y)
    with pytest.raises(ValueError, match="y must be"):
        ops.moe_lora_fwd(x, A, B, off, x)
    with pytest.raises(ValueError, match="accumulate"):
        ops.moe_lora_bwd(x, y, A, B, off, torch.zeros(4, 8), accumulate=True)


def test_block_norm_workspace_covers_what_the_backward_writes(lib):
    """At every width and many row counts the entry accepts the size its own query gives; it
    compares that size with the partial rows it would write (without a GPU the launch
    behind the checks is what fails; with one the entry is not called)."""
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    far = lambda i: (i + 1) << 36
    for dt, q in ((BF16, 8), (F32, 4)):
        for chunks in [*range(1, 1100, 7), 64, 65, 128, 129, 256, 257, 1024, 1025, 2048, 4096]:
            for T in (1, 255, 257, 1025, 2500, 20000):
                d = chunks * q
                nb = lib.moe_block_norm_bwd_workspace_size(T, d)
                a = _make(_lib.BlockNormBwdArgs, dtype=dt, T=T, d=d, res_scale=1.0, eps=1e-6,
                          h1=far(0), y=far(1), dh1=far(2), dx=far(3), w_post=far(4), w_pre=far(7),
                          dh=far(8), dy=far(9), dw_post=far(10), dw_pre=far(13), ws=far(14),
                          ws_bytes=nb)
                assert _status(lib.moe_block_norm_bwd, a) == _lib.MOE_ERR_HIP, (dt, d, T)
