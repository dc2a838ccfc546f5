"""Refusals that the header names, one by one (no GPU: they come before any device
call)."""

from tests.test_products_host import at, matmul, rows, shape

UNSUPPORTED, INVALID = -2, -1


def test_columns_side_by_side_are_refused():
    """A and C in the same rows of one array, and B and C: no byte is in both, but
    the addresses from first to last are."""
    m = shape("nt", groups=1, lda=64, ldc=64, group_stride=0)
    assert matmul(m, a=at(1), c=at(1, 80)) == INVALID
    m = shape("nt", groups=1, ldb=64, ldc=64, group_stride=0)
    assert matmul(m, b=at(2), c=at(2, 80)) == INVALID
    m = shape("tn", groups=1, lda=64, ldc=64, group_stride=0)
    assert matmul(m, a=at(1), c=at(1, 48)) == INVALID


def test_rows_of_codes_limits():
    assert rows(n=1 << 24) == UNSUPPORTED
    assert rows(cols=(1 << 30) + 1, ldx=1 << 31, ldc=1 << 31) == UNSUPPORTED
    assert rows(groups=65537) == UNSUPPORTED
