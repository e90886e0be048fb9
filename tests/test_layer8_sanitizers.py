"""The host-side checks of the router and the 8-bit operators in an address- and undefined-behaviour-sanitizer build (CPU)."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "comm_matmul_tensor_amd", "csrc")


def test_layer8_validation_under_asan_ubsan(tmp_path):
    exe = str(tmp_path / "driver")
    flags = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-g", "-O1"]
    sources = [os.path.join(CSRC, f) for f in ("validate_layer8.cpp", "validate_layer.cpp", "validate.cpp")]
    r = subprocess.run(["g++", "-std=c++17", *flags, f"-I{ROOT}/include", f"-I{CSRC}",
                        os.path.join(ROOT, "tests", "sanitize", "validate_layer8_driver.cpp"), *sources, "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = {k: v for k, v in os.environ.items() if k != "LD_PRELOAD"}
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0 and "clean" in r.stdout, (r.stdout + r.stderr)[-3000:]
