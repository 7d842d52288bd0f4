"""Launch and plan code of the operators beside the layer under AddressSanitizer and
UndefinedBehaviorSanitizer, CPU only: their sources' host parts are compiled with sanitizers and
linked with a stand-in for the runtime's calls, which checks the sizes of every launch."""
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_host_sanitizers import PKG, ROCM, ROOT, _tool

SOURCES = ("ops_api", "norm", "rms_norm", "quantize", "grouped", "grouped_f8", "orthogonalize",
           "orthogonalize_small", "balance_loss")


@pytest.fixture(scope="module")
def checks(tmp_path_factory):
    hipcc = _tool(os.path.join(ROCM, "bin", "hipcc"))
    clang = _tool(os.path.join(ROCM, "llvm", "bin", "clang++"))
    out = tmp_path_factory.mktemp("launches")
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer"]

    def compile_one(pair):
        src, obj = pair
        return obj, subprocess.run([hipcc, "--offload-arch=gfx950", "--offload-host-only", "-O1", "-g",
                                    "-std=c++17", "-fPIC", *san, "-I", os.path.join(ROOT, "include"),
                                    "-I", os.path.join(PKG, "csrc"), "-x", "hip", "-c", src, "-o", str(obj)],
                                   capture_output=True, text=True, timeout=600)

    pairs = [(os.path.join(PKG, "csrc", s + ".hip"), out / (s + ".o")) for s in SOURCES]
    pairs.append((os.path.join(ROOT, "tests", "sanitize", "launch_host_checks.cpp"), out / "checks.o"))
    with ThreadPoolExecutor(4) as ex:
        objects = []
        for obj, r in ex.map(compile_one, pairs):
            assert r.returncode == 0, r.stderr[-3000:]
            objects.append(str(obj))
    exe = out / "launch_host_checks"
    # (the objects name their device code, which a host-only compilation leaves out)
    r = subprocess.run([clang, "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fuse-ld=lld",
                        "-no-pie", "-Wl,--unresolved-symbols=ignore-all", *objects, "-o", str(exe)],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]

    def run(part):
        env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0",
                   UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
        r = subprocess.run([str(exe), part], capture_output=True, text=True, timeout=300, env=env)
        got = r.stdout + r.stderr
        assert "ERROR: AddressSanitizer" not in got and "runtime error" not in got, got[-4000:]
        assert r.returncode == 0 and "ALL OK" in r.stdout, got[-4000:]

    return run


@pytest.mark.parametrize("part", ["tiles", "balance", "products", "rows"])
def test_launches_and_plans(checks, part):
    checks(part)
