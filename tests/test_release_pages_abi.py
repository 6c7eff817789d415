"""Refusals of the page count of msa_release_pages, without a GPU."""
import pytest

from test_serving_abi import INV, abi, call, release_args  # noqa: F401


@pytest.mark.parametrize("num_pages", [-1, 1 << 31])
def test_num_pages_refused(abi, num_pages):  # noqa: F811
    assert call(abi, "msa_release_pages", release_args(abi, num_pages=num_pages)) == INV
    assert b"num_pages" in abi.load().msa_last_error_string()
