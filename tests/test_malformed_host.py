"""Page plans and adjustments on inputs that make no sense, in host builds of
the kernels' own sources whose arrays end at pages without access."""
import pytest

from tests import host_kernel


@pytest.mark.parametrize("source,edits", [("pages.hip", (('#include "device.hpp"', '#define PAGES\n#include "device.hpp"'),)),
                                          ("adjust.hip", ())])
def test_nothing_beyond_the_arrays_is_touched(tmp_path, source, edits):
    program = host_kernel.program(tmp_path, source, "malformed_host.cpp", edits)
    host_kernel.run(program, 0, 400)
