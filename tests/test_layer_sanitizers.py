"""The sequence-layer library's host code under AddressSanitizer and UndefinedBehaviorSanitizer (CPU).

As tests/test_abi_sanitizers.py does for the convolution's library: the
sources are rebuilt with the sanitizers on the host side only and the host
ABI suite (tests/test_layer_abi.py) runs against that build in a child
process that preloads the clang ASan runtime."""
import glob
import os
import subprocess
import sys
import textwrap

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "gated_convolution_sequence_amd", "csrc")
HIPCC = "/opt/rocm/bin/hipcc"

CHILD = textwrap.dedent('''
    import sys
    sys.path.insert(0, sys.argv[2]); sys.path.insert(0, sys.argv[2] + "/tests")
    import gated_convolution_sequence_amd as hc
    from gated_convolution_sequence_amd import layer
    hc.LAYER_LIB_PATH = layer.LAYER_LIB_PATH = sys.argv[1]   # the sanitized build
    import pytest
    sys.exit(pytest.main(["-q", "-x", "-m", "not gpu", "-p", "no:cacheprovider",
                          sys.argv[2] + "/tests/test_layer_abi.py"]))
''')


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")
def test_layer_abi_host_code_clean_under_asan_and_ubsan(tmp_path):
    found = sorted(glob.glob("/opt/rocm/llvm/lib/clang/*/lib/linux/libclang_rt.asan-x86_64.so"))
    if not found:
        pytest.skip("clang ASan runtime not installed")
    lib = str(tmp_path / "libhyena_layer_san.so")
    san = []
    for flag in ("-fsanitize=address", "-fsanitize=undefined", "-fno-omit-frame-pointer", "-shared-libsan"):
        san += ["-Xarch_host", flag]
    cmd = [HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-shared",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-I" + os.path.join(ROOT, "include")]
    cmd += san + ["-o", lib] + [os.path.join(CSRC, n) for n in ("hyena_scan.hip", "hyena_step.hip", "hyena_linear.hip")]
    subprocess.run(cmd, check=True, capture_output=True)
    logs = str(tmp_path / "san")
    env = dict(os.environ, LD_PRELOAD=found[-1],
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1:log_path=" + logs,
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1:log_path=" + logs)
    r = subprocess.run([sys.executable, "-c", CHILD, lib, ROOT], env=env, capture_output=True, text=True, timeout=600)
    reports = "".join(open(f).read() for f in glob.glob(logs + "*"))
    assert r.returncode == 0 and not reports, reports[-4000:] + r.stdout[-2000:] + r.stderr[-2000:]
    assert "passed" in r.stdout, r.stdout[-2000:]
