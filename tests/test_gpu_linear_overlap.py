"""Overlapping tensors through the Python face of the linear attention (marked gpu)."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu


def test_python_outputs():
    """Views of one buffer that overlap are refused, views that touch are not."""
    import torch
    import gated_delta_rule_71_amd as gdr
    n = 40 * 2 * 64
    buf = torch.randn(4 * n, device="cuda")
    view = lambda i: buf[i:i + n].view(1, 40, 2, 64)  # noqa: E731
    q, k, v, g = view(0), view(n), view(2 * n), torch.full((2,), -0.1, device="cuda")
    want, _ = gdr.chunk_linear_attention(q, k, v, g)
    with pytest.raises(RuntimeError):
        gdr.chunk_linear_attention(q, k, v, g, out=view(2 * n + 128))
    got, _ = gdr.chunk_linear_attention(q, k, v, g, out=view(3 * n))
    assert torch.equal(got, want)
    state = torch.zeros((40, 2, 64, 64), device="cuda")
    one = lambda i: view(i).view(40, 2, 64)  # noqa: E731
    with pytest.raises(RuntimeError):
        gdr.linear_attention_decode(one(0), one(n), one(2 * n), g, state, out=one(2 * n + 128))
    gdr.linear_attention_decode(one(0), one(n), one(2 * n), g, state, out=one(3 * n))
    # no tokens: rows of no bytes may lie anywhere
    none = buf[128:128].view(1, 0, 2, 64)
    final = buf[:2 * 64 * 64].view(1, 2, 64, 64)
    gdr.chunk_linear_attention(none, none, none, g, initial_state=state[:1], final_state=final)
    assert torch.equal(final, state[:1])
