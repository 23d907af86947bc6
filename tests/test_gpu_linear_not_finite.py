"""GPU gradients of the linear attention with NaN and infinities among their inputs (marked gpu):
rows that no such value reaches (the fp64 oracle's are finite there) have their values, the
others show it, over the borders of chunks and windows and for grouped heads.

Bounds of the rows that are not reached, with M the sum of the terms' magnitudes and
u = 2^-24: (L + 320) u M for the float32 sums (L tokens of carries and accumulation, products
over 128 channels, 64 scores), with bf16 inputs two roundings to 16 bits, 2^-15 M, and the last
rounding, 2^-8 of the result.
"""
from __future__ import annotations

import numpy as np
import pytest

from gated_delta_rule_71_amd import workloads as W
from oracle import linear_attention as LA
from parity import to_dev, to_host

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def rows_as(x, r, m, length, b16, what):
    x = to_host(x)
    clean = np.isfinite(r).all(-1)
    dirty = ~np.isfinite(x).all(-1)
    assert np.array_equal(dirty, ~clean), (what, np.argwhere(dirty == clean)[:4].tolist())
    tol = ((length + 320) * U + (2.0 ** -15 if b16 else 0)) * m + 1e-30
    if b16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(r)
    off = np.abs(x[clean] - r[clean]) / tol[clean]
    assert off.size == 0 or off.max() <= 1, f"{what}: {off.max():.3g} of the bound"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hk,Hv,K,V", [(2, 2, 128, 128), (2, 4, 64, 128)])
@pytest.mark.parametrize("lens", [[40, 150, 50], [70, 500, 31]])
def test_gradients(dtype, Hk, Hv, K, V, lens):
    import gated_delta_rule_71_amd as gdr
    T, N = sum(lens), len(lens)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    r = np.random.default_rng(5)
    st = W.BF16 if dtype == "bf16" else W.F32
    shapes = dict(q=(1, T, Hk, K), k=(1, T, Hk, K), v=(1, T, Hv, V), do=(1, T, Hv, V))
    x = {n: W.store(r.standard_normal(s, dtype=np.float32), st) for n, s in shapes.items()}
    s0, dht = r.standard_normal((2, N, Hv, K, V)).astype(np.float32)
    g = -np.exp2(-np.linspace(5, 9, Hv)).astype(np.float32)
    fin = {n: W.as_f64(a) for n, a in x.items()}
    mag = LA.backward(*(np.abs(fin[n]) for n in "qkv"), g, np.abs(fin["do"]), dht=np.abs(dht),
                      initial_state=np.abs(s0), cu_seqlens=cu)
    first, last = int(cu[1]), int(cu[2]) - 1
    for what, at, bad in (("v", 100, np.nan), ("q", last - 3, np.inf), ("do", last - 64, np.nan),
                          ("k", first, -np.inf), ("q", first + 63, np.nan), ("v", last, np.inf),
                          ("do", first, np.inf), ("k", last - 70, np.nan), ("dht", 1, np.nan),
                          ("s0", 1, np.inf)):
        dev = {n: to_dev(a) for n, a in x.items()}
        dev.update(s0=to_dev(s0), dht=to_dev(dht))
        f = {n: a.copy() for n, a in {**fin, "s0": s0, "dht": dht}.items()}
        place = (1, 1, 3, 7) if what in ("s0", "dht") else (0, at, 1, 5)
        dev[what][place] = float(bad)
        f[what][place] = bad
        got = gdr.chunk_linear_attention_backward(
            dev["q"], dev["k"], dev["v"], to_dev(g), dev["do"], dev["dht"],
            initial_state=dev["s0"], cu_seqlens=to_dev(cu))
        with np.errstate(invalid="ignore"):
            ref = LA.backward(f["q"], f["k"], f["v"], g, f["do"], dht=f["dht"],
                              initial_state=f["s0"], cu_seqlens=cu)
        for name, y, z, m in zip(("dq", "dk", "dv", "dh0"), got, ref, mag):
            if name == "dh0":   # a state at a time
                y, z, m = (a.reshape(N, Hv, K * V) for a in (y, z, m))
            rows_as(y, z, m, max(lens), dtype == "bf16" and name != "dh0",
                    f"{name}, {what} {bad} at {place}")
