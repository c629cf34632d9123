"""Workspace sizes of forks, by what the workspace holds: 16 bytes, a count and two
rows of the table for each sequence, a bit a page and a count for each 8192 pages."""
import pytest

from test_cache_abi import lib  # noqa: F401


@pytest.mark.parametrize("pages", [1, 8191, 8192, 8193, 70000, 2 ** 31 - 8193, 2 ** 31 - 8192, 2 ** 31 - 8191, 2 ** 31 - 1])
@pytest.mark.parametrize("B,width", [(1, 1), (2, 4), (300, 9), (65535, 32000)])
def test_forks(lib, pages, B, width):  # noqa: F811
    chunks = -(-pages // 8192)
    parts = (16 * B, 4 * B, 4 * B * width, 4 * B * width, 1024 * chunks, 4 * chunks)
    assert lib.fa_cache_fork_workspace_size(B, pages, width) == sum(-(-n // 256) * 256 for n in parts)
