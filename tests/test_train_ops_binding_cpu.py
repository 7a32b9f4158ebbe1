"""What the training operators' entry points and binding refuse or keep, on the host."""

import pytest

from nvfp4_mixture_experts_counting_gb300 import build as build_mod
from nvfp4_mixture_experts_counting_gb300 import ftmoe


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return ftmoe.lib()


def test_withhold_policy_limits(lib):
    for limit in (-1, 1_000_000_001):
        with pytest.raises(ftmoe.FtmoeError):
            ftmoe.ftmoe_test_withhold_policy(True, limit)
    ftmoe.ftmoe_test_withhold_policy(True, 1_000_000_000)
    ftmoe.ftmoe_test_withhold_policy(False)
