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


def test_gather_without_requests_needs_no_lengths(lib):  # noqa: F811
    """(Past the checks there is no device here, or a launch.)"""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are no device memory")
    assert lib.dn_kv_gather(*args("gather", B=0, kv=None, table=None)) != INVALID


def test_no_workspace_for_sizes_that_are_refused(lib):  # noqa: F811
    for B, total, heads, group in ((1, 4, 1 << 20, 2), (1, 1 << 28, 8, 1), (1, 1 << 28, 1, 8), (1, 1 << 27, 4, 4)):
        assert lib.dn_attn_paged(*args("attn", B=B, total=total, heads=heads, group=group, qs=heads * group * 64)) == INVALID
        assert lib.dn_attn_workspace_bytes(B, total, heads, group, 64) == 0
    assert lib.dn_attn_workspace_bytes(1, 1 << 28, 1, 4, 64) > 0
