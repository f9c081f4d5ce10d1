"""Host-only checks of sizes whose sums would leave 32 bits in the cache, attention and block-norm kernels: they are refused."""
import pytest

from test_block_abi import UNSUPPORTED, lib, norm  # noqa: F401

TOP = 2 ** 31 - 1


@pytest.mark.parametrize("rows", [TOP, TOP - 65535])
def test_norm_rows(lib, rows):  # noqa: F811
    """A CTA's next row is its row plus the grid."""
    assert norm(lib, rows=rows, dim=8) == UNSUPPORTED
