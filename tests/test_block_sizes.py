"""Host-only checks of sizes whose sums would leave 32 bits in the cache, attention and block-norm kernels: they are refused."""
import pytest

from test_block_abi import UNSUPPORTED, append, at, attend, lib, norm, workspace  # noqa: F401

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


@pytest.mark.parametrize("kw", [dict(n=2 ** 27, slots=at(15)), dict(T=2 ** 30, hkv=8, ks=1024, vs=1024, hq=8, qs=1024),
                                dict(T=2 ** 20, hkv=2, hq=2 ** 18, qs=2 ** 25)])
def test_append_work(lib, kw):  # noqa: F811
    """Blocks and query warps are counted in 32 bits; too many are a size that is not supported, not a failed launch."""
    assert append(lib, **kw) == UNSUPPORTED


def test_python_integers():
    """Values that do not fit a C int keep their meaning: nothing wraps round."""
    from gated_deltanet_linear_03_gb300.attn import _int32
    assert [_int32(x) for x in (0, 7, TOP, TOP + 1, 2 ** 32, 2 ** 32 + 5, -1, -2, -2 ** 31, -2 ** 32, -2 ** 40)] == \
        [0, 7, TOP, TOP, TOP, TOP, -1, -1, -1, -1, -1]
