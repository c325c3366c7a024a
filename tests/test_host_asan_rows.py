"""AddressSanitizer check of the host code of rows by group, adapters and draft verification.

Their sources are rebuilt with AddressSanitizer on the host code only (device code is
compiled as usual and never runs here); `host_asan_rows.cpp` drives the workspace sizes over
many shapes and the argument checks through it.
"""
import glob
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "two_sided_gptq_amd", "csrc")
SOURCES = ["common.hip", "groups.hip", "adapters.hip", "drafts.hip"]
ROCM = "/opt/rocm"


def test_host_code_of_rows_adapters_and_drafts_under_address_sanitizer(tmp_path):
    hip = os.path.join(ROCM, "bin", "hipcc")
    cxx = os.path.join(ROCM, "llvm", "bin", "clang++")
    rt = glob.glob(os.path.join(ROCM, "llvm", "lib", "clang", "*", "lib", "linux", "libclang_rt.asan-x86_64.so"))
    if not (os.path.exists(hip) and os.path.exists(cxx) and rt):
        pytest.skip("hipcc, clang++ or the AddressSanitizer runtime is missing")
    lib, drv = tmp_path / "libbakron_asan.so", tmp_path / "driver"
    inc = ["-I", os.path.join(ROOT, "include")]
    subprocess.run([hip, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-shared",
                    "-fhip-fp32-correctly-rounded-divide-sqrt", "-parallel-jobs=4",
                    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
                    "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fno-omit-frame-pointer",
                    *inc, "-I", CSRC, *[os.path.join(CSRC, s) for s in SOURCES], "-o", str(lib)],
                   check=True, capture_output=True, timeout=600)
    subprocess.run([cxx, "-std=c++17", "-O1", "-g", "-pthread", "-fsanitize=address", "-fno-omit-frame-pointer", *inc,
                    os.path.join(HERE, "host_asan_rows.cpp"), f"-L{tmp_path}", "-lbakron_asan",
                    f"-Wl,-rpath,{tmp_path}", f"-Wl,-rpath,{ROCM}/lib", "-o", str(drv)],
                   check=True, capture_output=True, timeout=300)
    r = subprocess.run([str(drv)], capture_output=True, text=True, timeout=600,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0"))
    print(r.stdout, r.stderr[-4000:])
    assert "AddressSanitizer" not in r.stderr
    assert r.returncode == 0 and "host checks passed" in r.stdout
