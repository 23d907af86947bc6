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


@pytest.mark.parametrize("heads,group", [(5, 96), (3, 640)])
def test_norm_rows_in_place(heads, group):
    """Outputs over the rows that they are made from, and a view shifted by one row refused."""
    import ctypes
    import torch
    import gated_delta_rule_71_amd as gdr
    from gated_delta_rule_71_amd import _lib
    lib = gdr.library()
    x, z, dy = torch.randn((3, 301, heads, group), device="cuda", dtype=torch.bfloat16)
    w, b = torch.randn((2, heads * group), device="cuda")
    want = gdr.group_norm_backward(x, w, dy, b, z=z)
    for over_dx, over_dz in (("dy", "z"), ("x", "dy"), ("z", "x")):
        t = dict(x=x.clone(), z=z.clone(), dy=dy.clone())
        dw, db = torch.empty_like(w), torch.empty_like(b)
        a = _lib.GroupNormBackwardArgs(301, heads, group, _lib.GDR_DTYPE_BF16, 1, 1e-5,
                                       t["x"].data_ptr(), t["z"].data_ptr(), w.data_ptr(),
                                       b.data_ptr(), t["dy"].data_ptr(), t[over_dx].data_ptr(),
                                       t[over_dz].data_ptr(), dw.data_ptr(), db.data_ptr())
        ws = torch.empty(lib.gdr_group_norm_backward_workspace_bytes(ctypes.byref(a)),
                         dtype=torch.uint8, device="cuda")
        a.workspace, a.workspace_bytes = ws.data_ptr(), ws.numel()
        assert lib.gdr_group_norm_backward(
            ctypes.byref(a), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
        for got, r in zip((t[over_dx], dw, db, t[over_dz]), want):
            assert torch.equal(got, r)
    buf = torch.randn((302, heads, group), device="cuda")
    with pytest.raises(RuntimeError):
        gdr.group_norm(buf[:-1], w, b, out=buf[1:])
