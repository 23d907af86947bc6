"""GPU linear attention with a decay per head: how many bits reach its outputs (marked gpu).

With bf16 inputs the matrix cores take bf16 operands, and a float32 value that meets them is
written in parts.  Rounding to bf16 is off by at most 2^-8 of the value, so two parts leave
2^-16 of it and three 2^-24.  The state and the scores have two parts where they meet q and v,
and so have the decayed values of a state that is not handed out.  Bounds, with u = 2^-24:
  * a result of ONE term (all other inputs zero, so that only exact zeros are added): 2^-16 of
    it for each two-part factor and at most (6 C + 14) u for its float32 factors, C the chunks
    of 64 tokens that it is carried over.  A carry or a border is a weight (expf and its
    correction, 4 u) and a product (u); the rest are a weight, its product with the value, the
    split, the products with q and k, the scales and the sums of the parts;
  * results of random inputs: each term's two-part roundings, at most two, fall either way, so
    that the result is off by at most sqrt(2) 2^-16 / sqrt(3) of its norm, and the (L + 320)
    float32 roundings of its sums by less than sqrt(2 (L + 320)) u: 2^-15 holds both;
  * a result rounded to bf16, against the reference rounded to bf16: an element that is off by
    d before rounding lands on the other side of a rounding border with probability
    d / step, then one step (at most 2^-7 of it) away, so that the mean square is at most
    d step: (2^-15 2^-7)^(1/2) = 2^-11 of the norm; 2^-10.5 leaves room for twice the mean.
"""
from __future__ import annotations

import numpy as np
import pytest

from gated_delta_rule_71_amd import workloads as W
from oracle import linear_attention as LA
from parity import to_dev, to_host

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def bf16(x):
    return W.store(np.asarray(x, np.float32), W.BF16)


def normal(seed, *shape):
    return bf16(np.random.default_rng(seed).standard_normal(shape, dtype=np.float32))


def one_term(x, r, bound, what):
    """Every element within ``bound`` of the reference's element; zeros are zeros.  Below 2^-126
    float32 has the spacing of 2^-126 itself, 2^-149, so that a rounding there is by at most
    2^-150 = 2^-126 u, and later weights are at most 1: the bound is taken of |r| + 2^-126."""
    x = to_host(x)
    assert x.shape == r.shape and np.all(np.isfinite(x)), what
    assert np.all(x[r == 0] == 0), what
    off = np.max(np.abs(x - r) / (np.abs(r) + 2.0 ** -126))
    assert off <= bound, f"{what}: {off / U:.1f} u, bound {bound / U:.1f} u"


def of_norm(x, r, bound, what):
    x = to_host(x)
    assert x.shape == r.shape and np.all(np.isfinite(x)), what
    off = np.linalg.norm(x - r) / np.linalg.norm(r)
    assert off <= bound, f"{what}: {off:.3g} of the norm, bound {bound:.3g}"


def rounded(r):
    return W.as_f64(bf16(r))


@pytest.mark.parametrize("K,V", [(64, 128), (128, 64), (128, 128)])
def test_state_meets_q(K, V):
    """o = scale lambda^(t+1) S0[row], one row of the state picked by a one-hot q."""
    import torch
    import gated_delta_rule_71_amd as gdr
    T, H = 130, 2
    g = np.array([-0.01, -0.2], np.float32)
    s0 = np.random.default_rng(1).standard_normal((1, H, K, V)).astype(np.float32)
    q = np.zeros((1, T, H, K), np.float32)
    q[0, np.arange(T), :, np.arange(T) * 7 % K] = 1.5
    zero = bf16(np.zeros((1, T, H, K)))
    o, _ = gdr.chunk_linear_attention(to_dev(bf16(q)), to_dev(zero),
                                      to_dev(bf16(np.zeros((1, T, H, V)))), to_dev(g),
                                      initial_state=to_dev(s0), out_dtype=torch.float32)
    r, _ = LA.prefill(q, 0 * q, np.zeros((1, T, H, V)), g, initial_state=s0)
    one_term(o, r, 2.0 ** -16 + (6 * 3 + 14) * U, "o")


@pytest.mark.parametrize("T,at", [(64, 3), (64, 60), (200, 70), (200, 3), (640, 300)])
def test_one_value(T, at):
    """v of one token alone: o_i = scale lambda^(i-at) (q_i . k) v, through the scores in the
    token's chunk and through the state behind it; q and k one-hot, so that q . k is a product."""
    import torch
    import gated_delta_rule_71_amd as gdr
    H, K, V = 2, 128, 128
    g = np.array([-0.002, -0.03], np.float32)
    q, v = np.zeros((1, T, H, K), np.float32), np.zeros((1, T, H, V))
    k = np.zeros_like(q)
    q[..., 5] = W.as_f64(normal(2, 1, T, H))
    k[0, at, :, 5] = 1.25
    v[0, at] = W.as_f64(normal(3, H, V))
    o, _ = gdr.chunk_linear_attention(to_dev(bf16(q)), to_dev(bf16(k)), to_dev(bf16(v)), to_dev(g),
                                      out_dtype=torch.float32)
    r, _ = LA.prefill(q, k, v, g)
    one_term(o, r, 2.0 ** -15 + (6 * -(-T // 64) + 14) * U, "o")


@pytest.mark.parametrize("Hk,Hv,K,V", [(2, 2, 128, 128), (1, 3, 64, 128), (1, 2, 128, 64)])
@pytest.mark.parametrize("lens", [[150], [300, 65, 700]])
def test_outputs_of_random_inputs(Hk, Hv, K, V, lens):
    """Outputs in float32 and bf16, slow and fast decays, with windows and without."""
    import torch
    import gated_delta_rule_71_amd as gdr
    T = sum(lens)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    q, k, v = normal(4, 1, T, Hk, K), normal(5, 1, T, Hk, K), normal(6, 1, T, Hv, V)
    g = -np.exp2(-np.linspace(3, 11, Hv)).astype(np.float32)
    s0 = np.random.default_rng(7).standard_normal((len(lens), Hv, K, V)).astype(np.float32)
    args = [to_dev(x) for x in (q, k, v, g)]
    r, _ = LA.prefill(*(W.as_f64(x) for x in (q, k, v)), g, initial_state=s0, cu_seqlens=cu)
    for final in (False, True):
        o = [gdr.chunk_linear_attention(*args, initial_state=to_dev(s0), cu_seqlens=to_dev(cu),
                                        output_final_state=final, out_dtype=t)[0]
             for t in (torch.float32, torch.bfloat16)]
        of_norm(o[0], r, 2.0 ** -15, "o, float32")
        of_norm(o[1], rounded(r), 2.0 ** -10.5, "o, bf16")


@pytest.mark.parametrize("Hk,Hv,K,V", [(2, 2, 128, 128), (1, 3, 64, 128), (1, 2, 128, 64)])
@pytest.mark.parametrize("lens", [[150], [300, 65, 700]])
def test_gradients_of_random_inputs(Hk, Hv, K, V, lens):
    import gated_delta_rule_71_amd as gdr
    T, N = sum(lens), len(lens)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    q, k = normal(14, 1, T, Hk, K), normal(15, 1, T, Hk, K)
    v, do = normal(16, 1, T, Hv, V), normal(17, 1, T, Hv, V)
    g = -np.exp2(-np.linspace(3, 11, Hv)).astype(np.float32)
    s0, dht = np.random.default_rng(18).standard_normal((2, N, Hv, K, V)).astype(np.float32)
    got = gdr.chunk_linear_attention_backward(
        *(to_dev(x) for x in (q, k, v, g, do, dht)), initial_state=to_dev(s0),
        cu_seqlens=to_dev(cu))
    ref = LA.backward(*(W.as_f64(x) for x in (q, k, v)), g, W.as_f64(do), dht=dht,
                      initial_state=s0, cu_seqlens=cu)
    for name, x, r in zip(("dq", "dk", "dv"), got, ref):
        of_norm(x, rounded(r), 2.0 ** -10.5, name)


def far_value(seed, T, H, D, at):
    """Rows of which one has values (its head's value channels, or one q/k channel of 1)."""
    x = np.zeros((1, T, H, D))
    x[0, at] = W.as_f64(normal(seed, H, D))
    return x


@pytest.mark.parametrize("K,V", [(64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("T,at", [(1, 0), (64, 2), (200, 3), (300, 100), (320, 1)])
def test_state_of_far_tokens(K, V, T, at):
    """k and v of one token alone, zeros behind it (a prompt padded at its end): the final
    state is that token's term, however far its weight has fallen.  In batched rows, a packed
    slot cache with other sequences around it, and for the gradient of the initial state."""
    import torch
    import gated_delta_rule_71_amd as gdr
    H = 3
    g = np.array([-0.002, -0.06, -0.25], np.float32)
    k, v = far_value(21, T, H, K, at), far_value(22, T, H, V, at)
    q = W.as_f64(normal(23, 1, T, H, K))
    bound = (6 * -(-T // 64) + 14) * U
    d = [to_dev(bf16(x)) for x in (q, k, v)]
    _, fs = gdr.chunk_linear_attention(*d, to_dev(g), output_final_state=True)
    _, r = LA.prefill(q, k, v, g)
    one_term(fs, r, bound, "final state")

    other = [to_dev(normal(s, 1, 70, H, n)) for s, n in ((24, K), (25, K), (26, V))]
    packed = [torch.cat([y, x, y], 1) for x, y in zip(d, other)]
    cu = torch.tensor([0, 70, 70 + T, 140 + T], dtype=torch.int32, device="cuda")
    cache = torch.zeros((4, H, K, V), device="cuda")
    slots = torch.tensor([3, 1, 0], dtype=torch.int32, device="cuda")
    gdr.chunk_linear_attention(*packed, to_dev(g), initial_state=cache, cu_seqlens=cu,
                               state_indices=slots)
    one_term(cache[1:2], r, bound, "slot")

    # back in time: q and do of one token alone, zeros before it
    qf, do = k[:, ::-1], v[:, ::-1]
    *_, dh0 = gdr.chunk_linear_attention_backward(
        to_dev(bf16(qf)), d[0], to_dev(normal(27, 1, T, H, V)), to_dev(g), to_dev(bf16(do)))
    *_, r = LA.backward(qf, q, np.zeros((1, T, H, V)), g, do)
    one_term(dh0, r, bound, "dh0")


@pytest.mark.parametrize("K,V", [(64, 128), (128, 128)])
def test_states_padded_with_zeros(K, V):
    """Random tokens, then zeros, as in rows that are filled up: float32 sums of at most two
    chunks of terms (each within 26 u of itself), then carries of 5 u each."""
    import gated_delta_rule_71_amd as gdr
    T, real, H = 320, 120, 2
    g = np.array([-0.01, -0.05], np.float32)
    q, k, v = (W.as_f64(normal(s, 1, T, H, n)) for s, n in ((31, K), (32, K), (33, V)))
    k[:, real:], v[:, real:] = 0, 0
    _, fs = gdr.chunk_linear_attention(*(to_dev(bf16(x)) for x in (q, k, v)), to_dev(g),
                                       output_final_state=True)
    _, r = LA.prefill(q, k, v, g)
    of_norm(fs, r, (26 + 6 * 5) * U / 3 ** 0.5, "final state")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 2])
def test_state_of_a_decoded_token(dtype, T):
    """lambda S + k v: expf (2 u), its product and the fused sum (u each), of T tokens."""
    import gated_delta_rule_71_amd as gdr
    n, H, K, V = 3, 2, 128, 64
    r = np.random.default_rng(41)
    q, k, v = (W.store(r.standard_normal((n, T, H, d), dtype=np.float32),
                       W.BF16 if dtype == "bf16" else W.F32) for d in (K, K, V))
    g = np.array([-0.3, -4.0], np.float32)
    cache = r.standard_normal((n, H, K, V)).astype(np.float32)
    d = to_dev(cache)
    gdr.linear_attention_decode(*(to_dev(x if T > 1 else x[:, 0]) for x in (q, k, v)), to_dev(g), d)
    f = [W.as_f64(x) for x in (q, k, v)]
    _, after, _ = LA.decode(*f, g, cache, np.arange(n))
    _, m, _ = LA.decode(*map(np.abs, f), g, np.abs(cache), np.arange(n))
    assert np.all(np.abs(to_host(d) - after) <= 4 * T * U * m)
