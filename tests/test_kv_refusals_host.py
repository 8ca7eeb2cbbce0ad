"""More of what the paged cache calls refuse on the host, before any device work. These run without a GPU."""
import math

import pytest

from test_kv_abi_host import attn, lib, pytestmark  # noqa: F401


@pytest.mark.parametrize("dtype,cache", [(0, 0), (0, 2), (0, 3), (1, 1), (1, 3)])
@pytest.mark.parametrize("scale", [math.nan, math.inf, -math.inf])
def test_a_scale_that_is_not_finite(lib, scale, dtype, cache):  # noqa: F811
    assert attn(lib, scale=scale, dtype=dtype, cache=cache) == -1
