"""What an output of the MXFP4 routed-expert layer may differ by from its
64-bit definition (tests/mx_reference.py), element by element, and inputs for
which that is little.

The inputs' scale bytes lie so close together that every sum of the gate/up
product is a whole number of quanta (the product of the operands' least scales
times a quarter) below 2^20 of them in magnitude, in any order: fp32 holds
them all, and the sums are exact.  What remains:
  silu      g * rcp(1 + exp2(-log2(e) g)) * u: the exponent's rounding and
            constant 1.25 |g| 2^-24, the exponential and the reciprocal one
            ulp (2^-23) each, the sum and two products 2^-24 each, so below
            (2 |g| + 8) 2^-24 relative.
  h         an h closer than that to a border of bf16 may take the other
            value, and only if a border of the E2M1 grid (or of its block's
            scale) lies between the two does its MXFP4 value change: `flip`
            is by how much.
  products  h^ W2^T: exact by the same count of quanta, or I * 2^-23 of the
            sum of magnitudes (2^-23: the matrix units may truncate).
  sum       at most 2 top_k + 16 roundings of 2^-24 (weights, slots in order, a
            workgroup's waves) of the sum of magnitudes.
  output    one rounding to bf16, half a step: 2^-8 relative.
"""
from __future__ import annotations

import numpy as np

import workloads as wl
from tests import mx_reference as ref


def experts_case(seed, T, E, k, H, I, skip=0.0, skew=0):
    """x, ids, weights, W13, W2 as for the layer; gate and up of about 2 rms.
    skew: that many of the tokens all take expert 0 first."""
    rng = np.random.default_rng(seed)
    x = wl.normal_bf16(rng, (T, H), 1.0)
    if k <= E:
        ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    else:
        ids = rng.integers(0, E, (T, k), dtype=np.int32)
    ids[:skew, 0] = 0
    if skip:
        ids[rng.random((T, k)) < skip] = -1
    tw = (rng.random((T, k)) + 0.25).astype(np.float32)
    lo = 127 + int(round(np.log2(0.7 / np.sqrt(H))))            # a code is 2.9 rms
    w13 = ref.random_mx(rng, E, 2 * I, H, lo=lo, hi=lo + 2)
    w2 = ref.random_mx(rng, E, H, I, lo=119, hi=121)
    return x, ids, tw, w13, w2


def quantum(codes, scales):
    """Per row: half the least scale of a block that holds anything."""
    some = (codes.reshape(*scales.shape, 16) & 0x77).any(axis=-1)
    return np.exp2(np.where(some, scales, 254).astype(np.float64).min(axis=-1) - 128.0)


def sum_error(a, aq, w, wq):
    """|a| |w|^T and what an fp32 sum of a w^T may be off by, in any order."""
    mag = np.abs(a) @ np.abs(w).T
    exact = mag < 2.0 ** 20 * aq[:, None] * wq[None, :]
    return mag, np.where(exact, 0.0, a.shape[1] * 2.0 ** -23 * mag)


def _encode_as(v, s):
    """Magnitudes v >= 0 [R, B, 32] under the scale bytes s [R, B], decoded."""
    q = v / np.exp2(s - 127.0)[..., None]
    mid = (ref.E2M1[:-1] + ref.E2M1[1:]) / 2
    code = np.zeros(q.shape, np.int64)
    for i in range(7):
        code += (q > mid[i]) | ((q == mid[i]) & (i % 2 == 1))
    return ref.E2M1[code] * np.exp2(s - 127.0)[..., None]


def _scale(amax):
    _, e = np.frexp(np.where(amax > 0, amax, 1.0))
    return np.where(amax > 0, np.clip(e - 3 + 127, 0, 254), 0).astype(np.float64)


def requantize(h, rel):
    """h (64 bits) -> its MXFP4 values, their quanta per row, and what each may
    differ by when h is off by rel relative."""
    R, I = h.shape
    bits = ref.bf16_round(h)
    packed = ref.mx_encode(bits)
    nominal = ref.mx_decode(*packed)
    a = np.abs(h)
    lo, hi = (ref.bf16_values(ref.bf16_round(v)).reshape(R, I // 32, 32) for v in (a * (1 - rel), a * (1 + rel)))
    s_lo, s_hi = _scale(lo.max(axis=2)), _scale(hi.max(axis=2))
    n = np.abs(nominal).reshape(R, I // 32, 32)
    flip = np.zeros_like(n)
    for v in (lo, hi):
        for s in (s_lo, s_hi):
            flip = np.maximum(flip, np.abs(_encode_as(v, s) - n))
    return nominal, quantum(*packed), flip.reshape(R, I)


def experts(x, ids, tw, w13, w2):
    """(out, bound): the layer in 64 bits and what each element may be off by.
    Asserts that the gate/up sums are exact, as the bound's smallness needs."""
    T, H = x.shape
    I = w2[0].shape[-1] * 2
    xp = ref.mx_encode(x)
    xh, xq = ref.mx_decode(*xp), quantum(*xp)
    out, slack, mags = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))
    for e in range(w13[0].shape[0]):
        t, j = np.nonzero(ids == e)
        if not t.size:
            continue
        w = ref.mx_decode(w13[0][e], w13[1][e])
        _, off = sum_error(xh[t], xq[t], w, quantum(w13[0][e], w13[1][e]))
        assert (off == 0).all(), "gate/up sums are not exact"
        gu = xh[t] @ w.T
        g, u = gu[:, :I], gu[:, I:]
        assert np.abs(g).max() < 80.0
        hh, hq, flip = requantize(g / (1.0 + np.exp(-g)) * u, (2 * np.abs(g) + 8) * 2.0 ** -24)
        w = ref.mx_decode(w2[0][e], w2[1][e])
        mag, off = sum_error(hh, hq, w, quantum(w2[0][e], w2[1][e]))
        c = tw[t, j, None].astype(np.float64)
        np.add.at(out, t, (hh @ w.T) * c)
        np.add.at(mags, t, mag * c)
        np.add.at(slack, t, (off + flip @ np.abs(w).T * (1 + 2.0 ** -10)) * c)
    slack += (2 * ids.shape[1] + 16) * 2.0 ** -24 * mags
    return out, slack + 2.0 ** -8 * (np.abs(out) + slack)


def check(y, want, bound):
    """y as float64 [T, H]."""
    assert np.isfinite(y).all()
    err = np.abs(y - want)
    bad = err > bound
    assert not bad.any(), (f"{bad.sum()} of {y.size} outside the bound, rows {np.unique(np.nonzero(bad)[0])[:8]}, "
                           f"up to {np.max(err[bad] / np.maximum(bound[bad], 1e-300)):.3g} times")
