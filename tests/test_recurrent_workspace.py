"""Host checks of the gated recurrence's workspace: a part of the rate's gradient for each block of a cluster, and a row of
few tokens has few."""
import pytest

from diagonal_state_space_gb300 import _native, build

TILE, CLUSTER = 32, 16                   # tokens of a backward tile, blocks of the largest cluster


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _native.lib()


@pytest.mark.parametrize("L", [0, 1, TILE, TILE + 1, 3 * TILE, CLUSTER * TILE, CLUSTER * TILE + 1, 1 << 20])
def test_parts_of_as_many_tiles_as_a_row_has(lib, L):
    parts = min(CLUSTER, max(1, -(-L // TILE)))
    for B, C in ((1, 8), (3, 77), (1000, 4096)):
        assert lib.s5_gated_scan_workspace_size(B, L, C) == 256 + 4 * B * parts * C
    assert lib.s5_gated_scan_workspace_size(0, L, 8) == 256
