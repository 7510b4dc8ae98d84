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


@pytest.mark.parametrize("sizes", [dict(num_rows=2 ** 31), dict(num_rows=2 ** 32 + 4), dict(num_rows=-1),
                                   dict(page_size=2 ** 32 + 16), dict(page_size=-2 ** 32 + 16)])
def test_sizes_are_not_taken_modulo_2_to_the_32(sizes):
    import torch
    import draft_token_verification_packed_amd as vsv
    i = lambda n: torch.zeros(n, dtype=torch.int32)
    with pytest.raises(ValueError, match="2\\^31"):
        vsv.plan_pages(i(4).view(1, 4), i(1), i(1), i(2), i(9), i(1), **dict(dict(page_size=16, num_rows=4), **sizes))
