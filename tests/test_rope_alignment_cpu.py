"""Positions that are not aligned to their 4 bytes are refused before any launch."""
import pytest

from gated_deltanet_recurrent_gb300 import abi
from tests.test_rope_cpu import call, lib  # noqa: F401  (a fixture)


@pytest.mark.parametrize("positions", [0x1001, 0x1002, 0x1003])
def test_positions(lib, positions):  # noqa: F811
    rope = abi.Rope(64)
    assert call(lib, rope.handle, positions=positions) == "GDN_ERR_ARG"
    assert "aligned" in lib.gdn_last_error_message().decode()
