"""The host side of the Muon step under AddressSanitizer and
UndefinedBehaviorSanitizer (no GPU): random units' tables cover every tile,
chunk and element once and stay inside the workspace, and the entry points
run up to their first launch, which reports that there is no device."""

import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CSRC = os.path.join(ROOT, "fully_sharded_amd", "csrc")
SOURCES = [os.path.join(CSRC, f) for f in ("plan.cpp", "abi.cpp", "graph.cpp", "muon.cpp")] + \
    [os.path.join(ROOT, "tests", "c", f)
     for f in ("launch_stub.cpp", "muon_launch_stub.cpp", "muon_sanitize.cpp")]
SAN = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
       "-Xarch_host", "-fno-sanitize-recover=all"]


def test_random_units_under_sanitizers(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("no hipcc")
    objs = []
    for src in SOURCES:
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        subprocess.run([HIPCC, "-x", "hip", "--offload-arch=gfx950", "-O1", "-g", "-std=c++17",
                        "-fno-omit-frame-pointer", *SAN, "-I", os.path.join(ROOT, "include"),
                        "-I", CSRC, "-c", src, "-o", obj], check=True, capture_output=True)
        objs.append(obj)
    exe = str(tmp_path / "muon_sanitize")
    subprocess.run([HIPCC, "--offload-arch=gfx950", *SAN[:4], *objs, "-o", exe, "-L/opt/rocm/lib",
                    "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib"], check=True, capture_output=True)
    out = subprocess.run([exe, "400"], capture_output=True, text=True, timeout=600,
                         env=dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
                                  UBSAN_OPTIONS="print_stacktrace=1"))
    assert "Sanitizer" not in out.stderr and "runtime error" not in out.stderr, out.stderr[-4000:]
    assert out.returncode == 0, (out.stdout[-3000:], out.stderr[-2000:])
    assert "checked 400 random units, failures 0" in out.stdout
