"""The host checks of the block norms, the gradient norm and the adapters under
AddressSanitizer, on the CPU: their sources compiled for the host only, linked with
tests/abi_block_asan_driver.cpp, whose calls are all refused before a launch."""
import concurrent.futures as cf
import os
import subprocess

import pytest

# (the compilers' flags and the stubs are its; a tree for GPU runs may come without it)
pytest.importorskip("test_abi_asan")
from test_abi_asan import ASAN, CLANG, CSRC, HERE, HIPCC, HOST_ASAN, ROOT, _fatbin_stubs  # noqa: E402


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)),
                    reason="needs the ROCm compilers")
def test_block_host_checks_under_asan(tmp_path):
    def compile_one(name):
        obj = str(tmp_path / (name + ".o"))
        _run([HIPCC, "--offload-arch=gfx950", "--offload-host-only", "-std=c++17", "-fPIC",
              *HOST_ASAN, "-c", os.path.join(CSRC, name), "-o", obj])
        return obj

    # (route.hip holds the count of compute units)
    with cf.ThreadPoolExecutor(max_workers=4) as ex:
        objs = list(ex.map(compile_one, ["norm.hip", "clip.hip", "lora.hip", "route.hip"]))
    stubs, drv, stub_o, exe = (str(tmp_path / n) for n in ("stubs.s", "driver.o", "stubs.o", "driver"))
    assert _fatbin_stubs(objs, stubs) == len(objs)
    _run([CLANG, "-std=c++17", *ASAN, "-I", os.path.join(ROOT, "include"), "-c",
          os.path.join(HERE, "abi_block_asan_driver.cpp"), "-o", drv])
    _run([CLANG, "-c", stubs, "-o", stub_o])
    _run([CLANG, *ASAN, drv, stub_o, *objs, "-L/opt/rocm/lib", "-lamdhip64",
          "-Wl,-rpath,/opt/rocm/lib", "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, (r.stdout[-3000:], r.stderr[-6000:])
    assert "abi host checks passed" in r.stdout
