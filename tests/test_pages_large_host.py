"""Page plans over 2^31 - 1 rows, in a host build of the kernel: a step over
the rows that passes 2^31 must end the loop, not reach before the array."""
import pytest

from tests import host_kernel


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    return host_kernel.program(tmp_path_factory.mktemp("pages"), "pages.hip", "pages_host.cpp")


@pytest.mark.parametrize("requests", [3, 300])
def test_rows_up_to_the_largest_number(program, requests):
    assert "ok" in host_kernel.run(program, requests)
