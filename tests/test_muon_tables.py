"""Which tiles the products of a unit get, and how many parts A's sums come in
(no GPU): the rules that choose between the kernels' forms."""

import os
import subprocess
from collections import namedtuple

import pytest

from tests.muon_units import UNITS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CSRC = os.path.join(ROOT, "fully_sharded_amd", "csrc")
SOURCES = [os.path.join(CSRC, f) for f in ("plan.cpp", "abi.cpp", "graph.cpp", "muon.cpp")] + \
    [os.path.join(ROOT, "tests", "c", f)
     for f in ("launch_stub.cpp", "muon_launch_stub.cpp", "muon_tables.cpp")]
Choice = namedtuple("Choice", "gram poly step longest parts")


@pytest.fixture(scope="module")
def choices(tmp_path_factory):
    """f([(rows, columns), ...]) -> the Choice for bf16 results, for fp32 ones."""
    if not os.path.exists(HIPCC):
        pytest.skip("no hipcc")
    exe = str(tmp_path_factory.mktemp("tables") / "muon_tables")
    subprocess.run([HIPCC, "-x", "hip", "--offload-arch=gfx950", "-O1", "-std=c++17", "-I",
                    os.path.join(ROOT, "include"), "-I", CSRC, *SOURCES, "-o", exe,
                    "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib"],
                   check=True, capture_output=True)

    def f(shapes):
        out = subprocess.run([exe], input=" ".join(f"{r} {c}" for r, c in shapes) + "\n",
                             capture_output=True, text=True, check=True, timeout=120).stdout
        v = [int(x) for x in out.split()]
        return Choice(*v[:5]), Choice(*v[5:])
    return f


LONG = 1 << 20


@pytest.mark.parametrize("shapes", [
    [(64, LONG), (1024, 1024)], [(32, LONG), (1024, 1024)], [(LONG, 40), (700, 700), (700, 900)],
    [(64, LONG // 2), (64, LONG // 2)] + [(512, 512)] * 2, [(100, 400000), (900, 900)]])
def test_a_long_matrix_beside_square_ones(choices, shapes):
    """A tile's parts are added up by one workgroup of 64 x 64 tiles, or three
    and more of 32 x 32: at most 32 parts for the larger ones, whatever else is
    in the unit."""
    for c in choices(shapes):
        assert c.gram == 32 or c.parts <= 32, c


@pytest.mark.parametrize("shapes,gram,parts", [
    ([(512, 29200)], 64, 15), ([(512, 32000)], 64, 16), ([(1024, 32000)], 64, 4),
    ([(32, LONG)], 32, 171), ([(64, LONG)], 32, 171), ([(512, 512)], 32, 1)])
def test_matrices_of_one_kind(choices, shapes, gram, parts):
    """Choices that were measured, each with its parts (two per compute unit
    at most, 32 rounds or more)."""
    bf16, _ = choices(shapes)
    assert bf16.gram == gram and bf16.parts <= parts and (bf16.parts > 1) == (parts > 1), bf16


@pytest.mark.parametrize("name", UNITS)
def test_units_that_take_each_tile(choices, name):
    """The units by which the kernels of every tile are tested get those tiles."""
    shapes, bf16, f32 = UNITS[name]
    got = choices(shapes)
    assert got[0][:3] == bf16 and got[1][:3] == f32
    assert got[0].parts <= 3


def test_every_tile_of_every_product_is_in_some_unit():
    for k in range(3):
        assert {u[1][k] for u in UNITS.values()} == {64, 128, 256}
        assert {u[2][k] for u in UNITS.values()} == {64, 128}


@pytest.mark.parametrize("shapes", [
    [(256, 500000), (600, 600)], [(320, 150000), (300, 300)], [(320, 600000), (300, 300)],
    [(256, LONG), (600, 600)], [(64, LONG), (320, 300000)]])
def test_long_matrices_whose_reading_outweighs_the_joining(choices, shapes):
    """64 x 64 tiles read A's operands half as often: with long matrices of
    more rows that is more than adding up a few dozen parts."""
    for c in choices(shapes)[0 if shapes[0][0] > 64 else 1:]:
        assert c.gram == 64, c
