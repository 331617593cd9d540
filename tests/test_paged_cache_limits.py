"""Sizes of the paged cache's workspace, and what its calls refuse, on the host alone (no GPU)."""

import pytest

from tests.test_paged_cache_abi import INVALID, NAMES, args, lib  # noqa: F401


def test_workspace_slots_begin_on_16_bytes(lib):  # noqa: F811
    """A partial result is read and written four floats at a time, also where a tile has an odd number of rows.

    Tiles of a batch have 2 * 152 + 64 slots.
    """
    for D in (64, 128, 256):
        for group in range(1, 129):
            assert lib.dn_attn_workspace_bytes(1, 64, 1, group, D) % (16 * (2 * 152 + 64)) == 0, (D, group)
