"""Refusals of a prefix call name the argument that is wrong (every check runs
before any CUDA call)."""
import pytest

from test_prefix_host import PREFIX
from test_serve_host import lib, refused  # noqa: F401


@pytest.mark.parametrize("change, code, msg", [
    (dict(pmax=0), -1, b"prefix_max_pages=0 must"),
    (dict(pmax=-3), -1, b"prefix_max_pages=-3 must"),
    (dict(n_groups=-1), -1, b"n_groups=-1 is negative"),
    (dict(pmax=1 << 28, n_groups=1), -2, b"prefix_max_pages * page_size = 4294967296"),
    (dict(pmax=1 << 20, n_groups=1 << 12), -2, b"n_groups * prefix_max_pages = 4294967296"),
    (dict(max_pages=0), -1, b"max_pages=0 must"),
])
def test_the_argument_is_named(lib, change, code, msg):  # noqa: F811
    refused(lib, lib.ra_paged_decode_prefix(*{**PREFIX, **change}.values()), code, msg)


def test_a_table_of_requests_is_not_called_a_prefix(lib):  # noqa: F811
    lib.ra_paged_decode_prefix(*{**PREFIX, "max_pages": 0}.values())
    assert b"prefix" not in lib.ra_last_error()
    lib.ra_paged_decode_prefix(*{**PREFIX, "max_pages": 1 << 30, "pmax": 0}.values())
    assert b"n_req * max_pages = 4294967296 exceeds" in lib.ra_last_error()
