"""CPU tests of the router's workspace sizes."""
import pytest

import gemm_epilogue_persistent_amd as gep
from gemm_epilogue_persistent_amd import _abi


def test_workspace_of_what_is_refused():
    """-1 for as many tokens as router_balance refuses whatever k is: 2^31 or more in all."""
    size = _abi.load().router_balance_workspace
    for batch, tokens in ((2, 1 << 30), (65535, 2 ** 31 - 1), (65535, 32769), (3, 715827883)):
        assert batch * tokens >= 1 << 31
        assert size(batch, tokens, 8) == -1
        with pytest.raises(ValueError):
            gep.router_balance_workspace(batch, tokens, 8)
    for batch, tokens in ((1, 2 ** 31 - 1), (65535, 32768), (3, 715827882), (2, 2 ** 30 - 1)):
        assert batch * tokens < 1 << 31
        assert size(batch, tokens, 8) > 0
