"""Helpers of the packed-sequence and paged-cache tests: seeded inputs, fp64 references sequence by
sequence through the oracle, and error bounds derived from the arithmetic.

Bounds. Rounding to bf16 is off by at most 2^-8 relative (half a step), to fp32 by 2^-24. A score is an
fp32 sum of d products in any order, so its error is at most delta = d 2^-23 scale max_ij sum_e |q_ie k_je|
(2^-23 per addition covers rounding toward zero). The exponential's argument, the exponential and the
logarithm add less than 2^-16 (arguments below 2^6 at 2^-24 each, exponentials at 2^-21). With
eps = delta + 2^-16:
  |LSE error| <= eps + 2^-22 |LSE|
  a probability is off by at most 2 eps relative (numerator and sum), and is rounded to bf16 before the
  product with V: |O error| <= 2^-8 |O| + (2^-8 + 2 eps + n 2^-23) (1 + 2^-8) sum_j P_ij |V_j|
  (n keys summed in fp32). The gradients follow the same way, in `grad_bounds`.
"""
from __future__ import annotations

import numpy as np

import oracle
import synth
from parity import bf16_tensor_to_f64, to_torch_bf16

U16 = 2.0 ** -8   # half a bf16 step, relative
SUM = 2.0 ** -23  # one fp32 addition, rounding toward zero included
EXP = 2.0 ** -16


def draw_packed(seed, ql, kl, Hq, Hkv, d):
    tq, tk = max(1, sum(ql)), max(1, sum(kl))
    return (synth.normal_bf16(seed, synth.STREAM_Q, (tq, Hq, d)), synth.normal_bf16(seed, synth.STREAM_K, (tk, Hkv, d)),
            synth.normal_bf16(seed, synth.STREAM_V, (tk, Hkv, d)))


def offsets(lens, start=0):
    import torch

    return torch.tensor(start + np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def sequences(ql, kl):
    """(query rows, key rows) of each sequence as slices."""
    q0 = k0 = 0
    for a, b in zip(ql, kl):
        yield slice(q0, q0 + a), slice(k0, k0 + b)
        q0, k0 = q0 + a, k0 + b


def score_error(q, k, scale):
    """delta above for one sequence ([n, H, d] fp64)."""
    if q.shape[0] == 0 or k.shape[0] == 0:
        return 0.0
    G = q.shape[1] // k.shape[1]
    top = max((np.abs(q[:, h]) @ np.abs(k[:, h // G]).T).max() for h in range(q.shape[1]))
    return q.shape[2] * SUM * scale * top


def reference(q, k, v, ql, kl, scale, causal):
    """O [Tq, Hq, d], LSE [Hq, Tq] and their bounds, all fp64, from the oracle."""
    O, L = np.zeros(q.shape), np.full((q.shape[1], q.shape[0]), -np.inf)
    bO, bL = np.zeros(q.shape), np.zeros(L.shape)
    for a, b in sequences(ql, kl):
        if a.stop == a.start or b.stop == b.start:
            continue
        n = b.stop - b.start
        eps = score_error(q[a], k[b], scale) + EXP
        o, l = oracle.attention(q[a][None], k[b][None], v[b][None], scale, causal)
        A, _ = oracle.attention(q[a][None], k[b][None], np.abs(v[b])[None], scale, causal)
        O[a], L[:, a] = o[0], l[0]
        bO[a] = U16 * np.abs(o[0]) + (U16 + 2 * eps + n * SUM) * (1 + U16) * A[0] + 1e-30
        bL[:, a] = eps + 2.0 ** -22 * np.where(np.isfinite(l[0]), np.abs(l[0]), 0)
    return O, L, bO, bL


def assert_within(got, want, bound, what):
    assert got.shape == want.shape, what
    assert np.all(np.isfinite(got)), f"{what}: non-finite values"
    over = np.abs(got - want) - bound
    assert over.max(initial=0.0) <= 0, \
        f"{what}: {np.count_nonzero(over > 0)} values over their bound, worst by {over.max():.3e}"


def assert_lse(got, want, bound, what):
    inf = np.isneginf(want)
    assert np.array_equal(np.isneginf(got), inf), f"{what}: -inf pattern of LSE differs"
    assert_within(got[~inf], want[~inf], bound[~inf], f"{what} LSE")


def grad_bounds(q, k, v, do, O, bO, ql, kl, scale, causal):
    """(dQ, dK, dV) in fp64 and their bounds. With e = 2 eps:
      dV = P^T dO: P off by e and rounded to bf16;
      dS = P (dP - D): P off by e, dP an fp32 sum of d products, D from the rounded O (off by bO), then
      rounded to bf16;  dQ = scale dS K,  dK = scale dS^T Q; each result rounded to bf16."""
    dQ, dK, dV = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    bQ, bK, bV = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    G, d = q.shape[1] // k.shape[1], q.shape[2]
    for a, b in sequences(ql, kl):
        nq, nk = a.stop - a.start, b.stop - b.start
        if nq == 0 or nk == 0:
            continue
        e = 2 * (score_error(q[a], k[b], scale) + EXP)
        r = oracle.attention_backward(q[a][None], k[b][None], v[b][None], do[a][None], scale, causal)
        dQ[a], dK[b], dV[b] = r[0][0], r[1][0], r[2][0]
        for h in range(q.shape[1]):
            g = h // G
            P = oracle.probabilities(q[a, h], k[b, g], scale, causal)
            dP = do[a, h] @ v[b, g].T
            D = (do[a, h] * O[a, h]).sum(1, keepdims=True)
            aO = np.abs(do[a, h])
            eD = (aO * bO[a, h]).sum(1, keepdims=True) + d * SUM * (aO * np.abs(O[a, h])).sum(1, keepdims=True)
            eP = d * SUM * (aO @ np.abs(v[b, g]).T)
            dS = P * (dP - D)
            E = (1 + U16) * (e * np.abs(dS) + P * (eD + eP)) + U16 * np.abs(dS)
            bV[b, g] += (U16 + e + nq * G * SUM) * (1 + U16) * (P.T @ aO)
            bQ[a, h] += scale * ((E + nk * SUM * np.abs(dS)) @ np.abs(k[b, g]))
            bK[b, g] += scale * ((E + nq * G * SUM * np.abs(dS)).T @ np.abs(q[a, h]))
    return (dQ, dK, dV), tuple(x + U16 * (np.abs(y) + x) + 1e-30 for x, y in ((bQ, dQ), (bK, dK), (bV, dV)))


f64 = synth.bf16_bits_to_f64
gpu = to_torch_bf16
host = bf16_tensor_to_f64
