"""The host code of the operators between a stage's boundary and its loss
(include/mapl_block.h) under AddressSanitizer and UndefinedBehaviorSanitizer on
the CPU, driven by tests/sanitize/block_driver.cpp.  Only host code is
instrumented; no kernel runs."""
import concurrent.futures as cf
import os
import subprocess

import pytest

from test_host_sanitizers import CSRC, ROOT, SAN, _hipcc


@pytest.mark.timeout(900)
def test_block_abi_under_address_and_undefined_behaviour_sanitizers(tmp_path):
    cc = _hipcc()
    if cc is None:
        pytest.skip("hipcc not available")
    import torch
    if torch.cuda.is_available():
        pytest.skip("a device is present: the driver's valid calls would launch kernels")
    common = ["-O1", "-g", "-std=c++17", "-fPIC", f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}"]
    sources = ["stage.hip", "fp8.hip", "attn.hip", "attn_bf16.hip", "distill.hip", "block_abi.hip"]
    # abi.hip has the device set-up, and takes the launchers of the rest
    from learned_activation_compression_amd.build import SOURCES

    def build(src):
        obj = str(tmp_path / src.replace(".hip", ".o"))
        # device code is never run here: only the host side of these operators' sources is instrumented
        san = SAN.split() if src in (*sources, "abi.hip") else []
        subprocess.run([cc, "--offload-arch=gfx950", *san, *common, "-c", os.path.join(CSRC, src), "-o", obj],
                       check=True, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
        return obj

    with cf.ThreadPoolExecutor(max_workers=8) as ex:
        objs = list(ex.map(build, SOURCES))
    drv, exe = str(tmp_path / "block_driver.o"), str(tmp_path / "block_driver")
    subprocess.run([cc, "-x", "c++", *SAN.split(), *common, "-I/opt/rocm/include", "-D__HIP_PLATFORM_AMD__", "-c",
                    os.path.join(ROOT, "tests", "sanitize", "block_driver.cpp"), "-o", drv], check=True,
                   stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    subprocess.run([cc, "--offload-arch=gfx950", *SAN.split(), *objs, drv, "-o", exe], check=True,
                   stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    p = subprocess.run([exe], env=env, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=300)
    assert p.returncode == 0, p.stdout[-4000:]
    assert "runtime error" not in p.stdout and "AddressSanitizer" not in p.stdout, p.stdout[-4000:]
    assert "all expectations held" in p.stdout
