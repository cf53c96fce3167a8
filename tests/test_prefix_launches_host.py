"""The two launches of a prefix call that overlap, by their source: the second
relies on the first, so they are made together, in one place."""
import re

from test_serve_edges_host import source


def test_the_shared_launch_directly_follows_the_own_one():
    api = source("serve_api.cu")
    assert api.count("kPagedShared") == 1 and api.count("kPagedOwn") == 1
    body = api[api.index("cudaError_t launch_apart("):]
    body = body[:body.index("\n}\n")]
    calls = re.findall(r"(?:ra::)?launch_\w+\(", body)[1:]
    assert calls == ["ra::launch_paged_decode("] * 2
    assert body.index("kPagedOwn") < body.index("kPagedShared")
    # Nowhere else is the kernel of the second launched.
    assert source("paged_kernel.cu").count("launch_paged_prefix(") == 1
    assert "launch_paged_prefix(" not in api


def test_modes_and_row_tiles_that_do_not_go_together_are_refused():
    kernel = source("paged_kernel.cu")
    body = kernel[kernel.index("cudaError_t launch_paged_decode("):]
    body = body[:body.index("\n}\n")]
    assert re.search(r"mode == kShared\) return row_tile == 128 \? .* : cudaErrorInvalidValue;", body)
    first = body.index("if (mode == kBoth && row_tile > 16) return cudaErrorInvalidValue;")
    assert first < body.index("launch_paged_tc(")
