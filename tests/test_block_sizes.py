"""Host-only checks of sizes whose sums would leave 32 bits in the cache, attention and block-norm kernels: they are refused."""
import pytest

from test_block_abi import UNSUPPORTED, attend, lib, norm, workspace  # noqa: F401

TOP = 2 ** 31 - 1


@pytest.mark.parametrize("rows", [TOP, TOP - 65535])
def test_norm_rows(lib, rows):  # noqa: F811
    """A CTA's next row is its row plus the grid."""
    assert norm(lib, rows=rows, dim=8) == UNSUPPORTED


@pytest.mark.parametrize("kv", [TOP, TOP - 62, TOP - 4095])
def test_attend_lengths(lib, kv):  # noqa: F811
    """A tile's last token is its first plus 64."""
    assert workspace(lib, mk=kv) == (0, UNSUPPORTED)
    assert workspace(lib, mk=kv, T=5000, mq=5000, d=256) == (0, UNSUPPORTED)
    assert attend(lib, mk=kv, max_pages=TOP, page=4096, n_pages=1) == UNSUPPORTED


def test_attend_lengths_below(lib):  # noqa: F811
    assert workspace(lib, mk=TOP - 4096)[1] == 0
