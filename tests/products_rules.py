"""The host side of the unit's products as a program: which kernel each gets, and
what the call returns where no GPU is."""

import os
import subprocess
from collections import namedtuple

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CSRC = os.path.join(ROOT, "fully_sharded_amd", "csrc")
SOURCES = [os.path.join(CSRC, f) for f in ("plan.cpp", "abi.cpp", "quant.cpp", "products.cpp")] + \
    [os.path.join(ROOT, "tests", "c", f)
     for f in ("launch_stub.cpp", "products_launch_stub.cpp", "products_rules.cpp")]
TILES = ["thin", "tiny", "apart", "small", "mid", "deep", "big"]
OPS = ["nt", "nn", "tn"]
TYPES = ["f32", "bf16", "i8"]
OK, INVALID, UNSUPPORTED, REACHED = 0, -1, -2, "the launch"
Rule = namedtuple("Rule", "tile direct parts status")


def build(directory):
    exe = os.path.join(str(directory), "products_rules")
    subprocess.run([HIPCC, "-x", "hip", "--offload-arch=gfx950", "-O1", "-std=c++17", "-I",
                    os.path.join(ROOT, "include"), "-I", CSRC, *SOURCES, "-o", exe,
                    "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib"],
                   check=True, capture_output=True)
    return exe


def rules(exe, products):
    """The Rule of each (op, type, groups, rows, n, k) or (..., lda, ldb, ldc,
    aligned)."""
    lines = []
    for p in products:
        op, kind, *rest = p
        rest = list(rest) + [0, 0, 0, 1][len(rest) - 4:]
        lines.append(" ".join(map(str, [OPS.index(op), TYPES.index(kind), *rest])))
    out = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True,
                         check=True, timeout=120).stdout.split("\n")
    got = []
    for line in out[:-1]:
        tile, direct, parts, status = map(int, line.split())
        got.append(Rule(TILES[tile], bool(direct), parts,
                        status if status in (OK, INVALID, UNSUPPORTED) else REACHED))
    assert len(got) == len(products)
    return got
