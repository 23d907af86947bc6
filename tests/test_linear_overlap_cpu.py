"""Arrays that may not overlap: the linear attention's and group norm's C entry points refuse
them before anything is enqueued (no GPU calls; addresses are never dereferenced)."""
from __future__ import annotations

import ctypes
import math

import pytest

from gated_delta_rule_71_amd import _lib

OK, INVALID = 0, 1
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def at(n):
    """Device addresses 64 MB apart, the first of them 64 MB."""
    return (n + 1) * 64 * MB


def args(struct, base, kw):
    a = struct()
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return a


def backward(**kw):
    """2 rows of 100 tokens, 4 heads of 128 x 64, bf16; states of 256 KB."""
    return args(_lib.LinearBackwardArgs, dict(
        batch=2, seqlen=100, num_seqs=2, num_qk_heads=4, num_v_heads=4, head_k=128, head_v=64,
        qkv_dtype=1, scale=math.nan, q=at(0), k=at(1), v=at(2), g=at(3), d_out=at(4), dq=at(5),
        dk=at(6), dv=at(7), initial_state=at(8), d_final_state=at(9), d_initial_state=at(10)), kw)


STATES = 4 * 2 * 4 * 128 * 64


@pytest.mark.parametrize("kw", [
    dict(d_initial_state=at(9)), dict(d_initial_state=at(8)),
    dict(d_initial_state=at(9) + STATES - 16), dict(d_initial_state=at(8) - STATES + 16),
    dict(d_initial_state=at(9), initial_state=0), dict(d_initial_state=at(8), d_final_state=0),
    dict(d_initial_state=at(9), seqlen=0)], ids=str)
def test_backward_states(lib, kw):
    """The gradient of the initial states is written while other workgroups read the states."""
    a = backward(**kw)
    assert lib.gdr_validate_linear_backward(ctypes.byref(a)) == INVALID
    assert lib.gdr_chunk_linear_attention_backward(ctypes.byref(a), None) == INVALID


@pytest.mark.parametrize("kw", [
    {}, dict(d_initial_state=at(9) + STATES), dict(d_initial_state=at(8) - STATES),
    dict(d_initial_state=0), dict(d_final_state=0, initial_state=0),
    dict(initial_state=at(9)), dict(d_initial_state=at(9), batch=0, num_seqs=0)], ids=str)
def test_backward_states_apart(lib, kw):
    assert lib.gdr_validate_linear_backward(ctypes.byref(backward(**kw))) == OK


def decode(**kw):
    """8 requests of 3 tokens, 4 heads of 128 x 64, bf16; 16 slots of 128 KB."""
    return args(_lib.LinearDecodeArgs, dict(
        batch=8, num_tokens=3, num_qk_heads=2, num_v_heads=4, head_k=128, head_v=64, num_slots=16,
        qkv_dtype=1, out_dtype=1, scale=math.nan, q=at(0), k=at(1), v=at(2), g=at(3), state=at(4),
        intermediate_state=at(5), out=at(6)), kw)


SLOT = 4 * 4 * 128 * 64


@pytest.mark.parametrize("kw", [
    dict(intermediate_state=at(4)), dict(intermediate_state=at(4) + 16 * SLOT - 16),
    dict(intermediate_state=at(4) - 8 * 3 * SLOT + 16),
    dict(intermediate_state=at(4) + SLOT, num_tokens=1)], ids=str)
def test_decode_states_between(lib, kw):
    """The states between the tokens would overwrite slots that other workgroups read."""
    assert lib.gdr_linear_attention_decode(ctypes.byref(decode(**kw)), None) == INVALID


@pytest.mark.parametrize("kw", [dict(intermediate_state=at(4) + 16 * SLOT),
                                dict(intermediate_state=at(4) - 8 * 3 * SLOT)], ids=str)
def test_decode_states_apart(lib, kw):
    a = decode(**kw)
    assert lib.gdr_validate_linear_decode(ctypes.byref(a)) == OK
    a.batch = 0
    assert lib.gdr_linear_attention_decode(ctypes.byref(a), None) == OK


def prefill(**kw):
    """2 rows of 400 tokens, 2/4 heads of 128 x 64, bf16: windows, and so a workspace."""
    a = args(_lib.LinearPrefillArgs, dict(
        batch=2, seqlen=400, num_seqs=2, num_qk_heads=2, num_v_heads=4, head_k=128, head_v=64,
        qkv_dtype=1, out_dtype=1, scale=math.nan, q=at(0), k=at(1), v=at(2), g=at(3), out=at(4),
        initial_state=at(5), final_state=at(6), workspace=at(7), workspace_bytes=32 * MB), kw)
    return a


ROWS = 2 * 400 * 2   # bytes of a bf16 channel of all tokens
QK, V = ROWS * 2 * 128, ROWS * 4 * 64


@pytest.mark.parametrize("kw", [
    dict(out=at(0) + QK - 16), dict(out=at(1) - V + 16), dict(out=at(2) + 512),
    dict(out=at(2) - 512), dict(out=at(2) - V, out_dtype=0), dict(out=at(3)),
    dict(out=at(5) + STATES - 16), dict(out=at(6)), dict(out=at(7) + 4096), dict(final_state=at(1)),
    dict(final_state=at(4) + 1024), dict(workspace=at(5)), dict(workspace=at(2) - 256)], ids=str)
def test_prefill_outputs(lib, kw):
    """Outputs (the workspace among them) that reach into an input or each other."""
    assert lib.gdr_chunk_linear_attention(ctypes.byref(prefill(**kw)), None) == INVALID


@pytest.mark.parametrize("kw", [
    dict(out=at(0) - 16), dict(out=at(1) + QK - 16), dict(out=at(2) + V - 64), dict(out=at(4) + SLOT),
    dict(out=at(4) + 16 * SLOT - 16), dict(out=at(5) + 16), dict(intermediate_state=at(0)),
    dict(intermediate_state=at(6) - 16 * SLOT), dict(state=at(1) - SLOT), dict(out=at(3))], ids=str)
def test_decode_outputs(lib, kw):
    kw = {**kw, "batch": 8, "num_tokens": 400 * 2 // 8}   # as many tokens as the prompts'
    assert lib.gdr_linear_attention_decode(ctypes.byref(decode(**kw)), None) == INVALID


@pytest.mark.parametrize("kw", [
    dict(dq=at(0) + 16), dict(dk=at(1) - 16), dict(dv=at(4) + 256), dict(dq=at(6) + 16),
    dict(dk=at(7) - 16), dict(dv=at(5) + 2 * 100 * 4 * 128 * 2 - 16), dict(dv=at(8)),
    dict(dk=at(9) + 32), dict(d_initial_state=at(2)), dict(d_initial_state=at(5)),
    dict(dq=at(3)), dict(num_qk_heads=2, workspace=at(4), workspace_bytes=32 * MB)], ids=str)
def test_backward_outputs(lib, kw):
    assert lib.gdr_chunk_linear_attention_backward(ctypes.byref(backward(**kw)), None) == INVALID


def test_outputs_apart(lib):
    """Arrays that touch, a state written in place, and arrays that are not given: past the
    checks (an empty batch, so that nothing is enqueued)."""
    for kw in ({}, dict(out=at(0) + QK), dict(out=at(2) - V), dict(final_state=at(5)),
               dict(final_state=0, initial_state=0), dict(out=at(5) + STATES)):
        assert lib.gdr_validate_linear_prefill(ctypes.byref(prefill(**kw))) == OK
    none = dict(batch=0, num_seqs=0)
    same = dict(out=at(0), final_state=at(0), initial_state=at(0))
    assert lib.gdr_chunk_linear_attention(ctypes.byref(prefill(**none, **same)), None) == OK
    assert lib.gdr_chunk_linear_attention_backward(ctypes.byref(backward(**none, dv=at(0))), None) == OK


def norm(**kw):
    """40 tokens of 3 x 64 channels, bf16."""
    return args(_lib.GroupNormArgs, dict(
        tokens=40, heads=3, group=64, dtype=1, activation=1, eps=1e-5, x=at(0), z=at(1),
        weight=at(2), bias=at(3), out=at(4)), kw)


def norm_backward(**kw):
    return args(_lib.GroupNormBackwardArgs, dict(
        tokens=40, heads=3, group=64, dtype=1, activation=1, eps=1e-5, x=at(0), z=at(1),
        weight=at(2), bias=at(3), dy=at(4), dx=at(5), dz=at(6), dweight=at(7), dbias=at(8),
        workspace=at(9), workspace_bytes=MB), kw)


NORM = 40 * 3 * 64 * 2


@pytest.mark.parametrize("kw", [
    dict(out=at(0) + 16), dict(out=at(0) - NORM + 16), dict(out=at(1) + NORM - 16),
    dict(out=at(2) + 4 * 192 - 16), dict(out=at(3)), dict(out=at(0) + NORM - 16, z=0)], ids=str)
def test_norm_output(lib, kw):
    """Rows shifted against the ones that are read (the same rows are worked in place)."""
    assert lib.gdr_group_norm(ctypes.byref(norm(**kw)), None) == INVALID


@pytest.mark.parametrize("kw", [
    dict(dx=at(0) + 16), dict(dx=at(4) - 16), dict(dx=at(1) + NORM - 16), dict(dz=at(5) + 16),
    dict(dz=at(0) + 384), dict(dweight=at(0)), dict(dweight=at(5) + 32), dict(dbias=at(7) + 16),
    dict(dbias=at(6)), dict(dx=at(2)), dict(workspace=at(4)), dict(workspace=at(5) + 1024),
    dict(workspace=at(7) - 4096)], ids=str)
def test_norm_gradients(lib, kw):
    assert lib.gdr_group_norm_backward(ctypes.byref(norm_backward(**kw)), None) == INVALID
