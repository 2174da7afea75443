"""The host checks of the 8-bit operand, product and loss calls (test_products_host.py)
against a build of the library's host code with AddressSanitizer and
UndefinedBehaviorSanitizer and stand-ins for the kernel launchers, in a child
process, as test_sanitized_host.py does for the other calls."""

import os
import shutil
import subprocess
import sys

from test_sanitized_host import CSRC, HOST_SOURCES, ROOT, _gxx


def test_products_host_tests_run_clean_under_asan_and_ubsan(tmp_path):
    gxx = _gxx()
    pkg = tmp_path / "tiled_movement_amd"
    pkg.mkdir()
    shutil.copy(os.path.join(ROOT, "tiled_movement_amd", "__init__.py"), pkg / "__init__.py")
    flags = ["-std=c++17", "-O1", "-g", "-fPIC", "-fno-omit-frame-pointer", "-fno-sanitize-recover=all",
             "-fsanitize=address,undefined", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
             f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}"]
    srcs = [os.path.join(CSRC, s) for s in HOST_SOURCES] + [os.path.join(ROOT, "tests", "host_stubs.cpp")]
    subprocess.run([gxx, *flags, "-shared", "-o", str(pkg / "libswz.so"), *srcs], check=True)
    runtimes = [subprocess.run([gxx, f"-print-file-name={n}"], capture_output=True, text=True).stdout.strip()
                for n in ("libasan.so", "libubsan.so")]
    env = dict(os.environ)
    env["LD_PRELOAD"] = " ".join(p for p in (*runtimes, env.get("LD_PRELOAD", "")) if p)
    env["ASAN_OPTIONS"] = "detect_leaks=0:halt_on_error=1:abort_on_error=0"
    env["UBSAN_OPTIONS"] = "halt_on_error=1:print_stacktrace=1"
    env["PYTHONPATH"] = os.pathsep.join([str(tmp_path), ROOT, env.get("PYTHONPATH", "")])
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-s", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_products_host.py")],
                       cwd=str(tmp_path), env=env, capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "ERROR: AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
