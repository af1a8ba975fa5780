"""The key/value cache's host code under AddressSanitizer and UndefinedBehaviorSanitizer, and its header as C99.

The C-ABI unit (csrc/kv.hip: argument checks, workspace sizes, launch parameters) is built beside csrc/w4a16.hip with
host code instrumented and the attention's launchers replaced by stand-ins (tests/sanitize/), and driven by the
host tests of the cache (tests/test_kv_host.py) in a child process.  tests/c_abi/kv_consumer.c uses
include/w4a16_kv.h from C99.
"""
import os
import shutil
import subprocess
import sys

import pytest

from test_sanitizers import HIPCC, ROOT, SAN, _env, _run, _runtime


def test_cache_abi_under_asan_ubsan(tmp_path):
    rt = _runtime()
    lib = str(tmp_path / "libw4a16_san.so")
    csrc = os.path.join(ROOT, "decode_w4a16_affine_amd", "csrc")
    cmd = [HIPCC, "--offload-arch=gfx950", "-x", "hip", "-std=c++17", "-fPIC", "-shared",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-I", os.path.join(ROOT, "include"), "-I", csrc,
           "-o", lib, os.path.join(csrc, "w4a16.hip"), os.path.join(csrc, "kv.hip"),
           os.path.join(ROOT, "tests", "sanitize", "host_stubs.hip"),
           os.path.join(ROOT, "tests", "sanitize", "kv_host_stubs.hip")]
    for f in SAN:   # host code only
        cmd[1:1] = ["-Xarch_host", f]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = _env(rt, W4A16_LIB=lib)
    probe = ("import decode_w4a16_affine_amd as w4; w4.kv_lib(); m = open('/proc/self/maps').read(); "
             f"assert {lib!r} in m and 'libclang_rt.asan' in m, 'instrumented library not loaded'")
    rc, out = _run([sys.executable, "-c", probe], env)
    assert rc == 0, out[-3000:]
    rc, out = _run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
                    os.path.join(ROOT, "tests", "test_kv_host.py")], env)
    assert rc == 0, out[-3000:]


def test_cache_header_from_c99(tmp_path):
    gcc = shutil.which("gcc")
    lib = os.path.join(ROOT, "decode_w4a16_affine_amd")
    if not gcc or not os.path.exists(os.path.join(lib, "libw4a16.so")):
        pytest.skip("gcc is not installed or libw4a16.so is not built")
    exe = str(tmp_path / "kv_consumer")
    r = subprocess.run([gcc, "-std=c99", "-O1", "-Wall", "-Wextra", "-Werror", "-pedantic",
                        "-I", os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "c_abi", "kv_consumer.c"),
                        "-o", exe, "-L", lib, "-lw4a16", "-L", "/opt/rocm/lib", "-lamdhip64",
                        f"-Wl,-rpath,{lib}:/opt/rocm/lib", "-Wl,--no-undefined"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.returncode, r.stdout, r.stderr)
