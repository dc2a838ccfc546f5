"""Which kernels the unit's products get (no GPU): the rules that choose between
their forms."""

import os

import pytest

from tests import products_rules as R
from tests.products_tiles import CASES


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    """f([(op, type, groups, rows, n, k), ...]) -> their Rules."""
    if not os.path.exists(R.HIPCC):
        pytest.skip("no hipcc")
    exe = R.build(tmp_path_factory.mktemp("rules"))
    return lambda products: R.rules(exe, products)


def test_cases_get_the_kernels_that_they_are_named_for(rules):
    """The products by which every kernel is tested on the GPU."""
    got = rules([(op, kind, len(sizes), sum(sizes), n, k, 0, 0, 0, int(off == 0))
                 for op, kind, sizes, n, k, off in CASES.values()])
    for name, r in zip(CASES, got):
        kind, op, tile, how = name.split()[:4]
        assert (kind, op) == (CASES[name][1], CASES[name][0]) and r.status == R.REACHED, name
        assert (r.tile, r.direct) == (tile, how == "direct"), (name, r)


def test_every_kernel_is_in_some_case():
    """As the launchers have them: thin and apart for products over rows, deep for
    bf16, and what passes through registers."""
    have = {tuple(name.split()[:4]) for name in CASES}
    tiles = {"bf16 direct": ["small", "mid", "deep", "big"], "i8 direct": ["small", "mid", "big"],
             "bf16 registers": ["small", "mid"], "f32 registers": ["tiny", "small", "mid"]}
    want = {(kind, op, tile, how) for key, all_of in tiles.items() for tile in all_of
            for kind, how in [key.split()] for op in R.OPS if (kind, op) != ("i8", "tn")}
    want |= {(kind, op, tile, "direct") for kind in ("bf16", "i8") for op in ("nt", "nn")
             for tile in ("thin", "apart")}
    assert have == want


@pytest.mark.parametrize("op", R.OPS)
def test_tiles_by_their_number(rules, op):
    """bf16 products of one weight with a sum of 2048, by their number of 128 x 128
    tiles: 64 x 64 ones up to half of the 256 compute units, where four times as
    many still run at once, deep ones up to all of them, shallow ones beyond.  No
    number stands alone."""
    def product(t):
        return (op, "bf16", 1, 2048, 128 * t, 2048) if op == "tn" else \
            (op, "bf16", 1, 128 * t, 2048, 2048)
    for down, r in zip(range(2, 24), rules([product(t) for t in range(2, 24)])):
        tiles = 16 * down
        want = {"deep"} if 128 < tiles <= 256 else {"mid"} if tiles > 256 else {"small", "apart"}
        assert r.tile in want, (tiles, r)
    # a few rows fewer or more do not change it
    near = [(op, "bf16", 1, 2048, x, 2048) if op == "tn" else (op, "bf16", 1, x, 2048, 2048)
            for x in (1920, 2000, 2040)]
    assert [r.tile for r in rules(near)] == ["deep"] * 3


@pytest.mark.parametrize("product,parts", [
    (("tn", "bf16", 150, 150 * 2048, 64, 64), 3), (("tn", "bf16", 200, 200 * 1024, 64, 128), 1),
    (("tn", "bf16", 200, 200 * 1024, 128, 128), 1), (("tn", "bf16", 130, 130 * 512, 128, 128), 1),
    (("nt", "bf16", 80, 80 * 64, 192, 4096), 1), (("nn", "bf16", 80, 80 * 64, 192, 4096), 1),
    (("nt", "bf16", 150, 150 * 40, 64, 4096), 1)])
def test_many_small_groups_keep_small_tiles(rules, product, parts):
    """Between half as many 128 x 128 tiles as compute units and one each, but of
    groups that fill little of them, or have few each."""
    r, = rules([product])
    assert r.tile in ("small", "thin", "apart") and r.parts == parts, r


def test_sums_in_parts_are_of_small_tiles(rules):
    """The joining launch is there for them alone."""
    products = [("tn", kind, groups, rows, n, k)
                for kind in ("f32", "bf16") for groups in (1, 3) for rows in (900, 40000)
                for n in (64, 200, 1000, 2000) for k in (8, 72, 1003, 2100)]
    got = rules(products)
    assert any(r.parts > 1 for r in got)
    for p, r in zip(products, got):
        assert r.parts == 1 or (r.tile == "small" and p[1] == "bf16"), (p, r)


LONG = 1 << 22   # entries: 8 MiB in bf16


@pytest.mark.parametrize("kind,groups,op,rows,n,k", [
    ("bf16", 1, "tn", 1, LONG, 8), ("bf16", 1, "tn", 1, 8, LONG + 1), ("bf16", 1, "nn", 3, LONG, 1),
    ("bf16", 5, "nn", 7, LONG + 3, 1), ("bf16", 1, "nt", 1, 1, LONG), ("f32", 1, "tn", 1, LONG, 3),
    ("f32", 2, "nn", 3, LONG, 1), ("f32", 1, "nt", 1, 1, LONG), ("bf16", 1, "nt", 1, 1, 1 << 25),
    ("i8", 1, "nn", 3, 1 << 23, 1)])
def test_operands_of_one_row_may_be_long(rules, kind, groups, op, rows, n, k):
    """Rows 8 MiB apart are refused; of one row nothing is apart, whatever the
    pitch is said to be."""
    far = 1 << 59 if kind == "i8" else (1 << 62) + 3
    lone_a = rows == 1
    lone_b = {"tn": rows, "nt": n, "nn": k}[op] == 1
    for lda in (0, far) if lone_a else (0,):
        for ldb in (0, far) if lone_b and groups == 1 else (0,):
            r, = rules([(op, kind, groups, rows, n, k, lda, ldb, 0, 1)])
            assert r.status == R.REACHED, (lda, ldb, r)


@pytest.mark.parametrize("op,rows,n,k", [("tn", 2, LONG, 8), ("tn", 2, 8, LONG),
                                         ("nn", 3, LONG, 2), ("nt", 1, 2, LONG),
                                         ("nt", 2, 1, LONG)])
def test_rows_far_apart_are_refused(rules, op, rows, n, k):
    at_most = (1 << 23) - 1
    assert [r.status for r in rules([
        (op, "bf16", 1, rows, n, k), (op, "f32", 1, rows, n, k),
        (op, "f32", 1, rows, min(n, at_most // 4), min(k, at_most // 4)),
        (op, "bf16", 1, rows, min(n, at_most // 2), min(k, at_most // 2))])] == \
        [R.UNSUPPORTED] * 2 + [R.REACHED] * 2
