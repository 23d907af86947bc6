"""Partial sums of the group norm's gradient: rows of them for as many token blocks as fill the
chip, whatever the number of heads (host only)."""
from __future__ import annotations

import pytest

import gated_delta_rule_71_amd as gdr


def blocks(tokens, heads, group):
    import torch
    x = torch.empty((tokens, heads, group), dtype=torch.bfloat16, device="meta")
    size = gdr.group_norm_backward_workspace_bytes(x)
    assert size % (2 * heads * group * 4) == 0
    return size // (2 * heads * group * 4)


@pytest.mark.parametrize("tokens,heads,group", [
    (1024, 512, 128), (2048, 32, 512), (64, 4096, 128), (300, 32, 512), (1 << 20, 60, 1024),
    (512, 65536, 64), (30000, 17, 128), (1, 4096, 1024)])
def test_wide_rows(tokens, heads, group):
    lanes = 4
    while lanes < 64 and 8 * lanes < group:
        lanes *= 2
    wide = -(-heads // min(heads, 256 // lanes))   # workgroups of a block of tokens
    n = blocks(tokens, heads, group)
    assert wide > 1 and 1 <= n and (n == 1 or n * wide <= 1024)


@pytest.mark.parametrize("tokens,heads,group,n", [(16384, 16, 128, 1024), (1501, 5, 96, 256),
                                                  (1, 4, 128, 1), (0, 4, 128, 1), (100, 16, 128, 100)])
def test_one_workgroup_a_block(tokens, heads, group, n):
    assert blocks(tokens, heads, group) == n
