"""Plain 64-bit definitions of the expert gate and of MXFP4, in numpy on the
host, for the parity tests; nothing here comes from the library."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


# ------------------------------------------------------------------- bf16 --

def bf16_values(bits: np.ndarray) -> np.ndarray:
    return (np.ascontiguousarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def bf16_round(x: np.ndarray) -> np.ndarray:
    """float64 -> bf16 patterns, to nearest even, rounded once (finite)."""
    x = np.asarray(x, np.float64)
    _, e = np.frexp(np.abs(x))                       # |x| = m 2^e, 1/2 <= m < 1
    step = np.exp2(np.maximum(e, -125) - 8.0)        # 8 significant bits, the least step 2^-133
    v = (np.rint(x / step) * step).astype(np.float32)  # exact in fp32
    return (v.view(np.uint32) >> 16).astype(np.uint16)


# ------------------------------------------------------------------ MXFP4 --

def mx_encode(bits: np.ndarray):
    """bf16 patterns [R, C] -> (codes uint8 [R, C/2], scale bytes [R, C/32])."""
    R, C = bits.shape
    v = bf16_values(bits).reshape(R, C // 32, 32)
    bad = ~np.isfinite(v).all(axis=2)
    a = np.where(np.isfinite(v), np.abs(v), 0.0)
    amax = a.max(axis=2)
    _, e = np.frexp(np.where(amax > 0, amax, 1.0))
    s = np.where(amax > 0, np.clip(e - 1 - 2 + 127, 0, 254), 0)
    q = a / np.exp2(s - 127.0)[..., None]
    mid = (E2M1[:-1] + E2M1[1:]) / 2
    code = np.zeros(q.shape, np.uint8)
    for i in range(7):                               # past a midpoint, or on it if the code above is even
        code += (q > mid[i]) | ((q == mid[i]) & (i % 2 == 1))
    code |= (np.signbit(v).astype(np.uint8) << 3)
    code = code.reshape(R, C)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8), np.where(bad, 255, s).astype(np.uint8)


def mx_decode(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    c = np.stack([codes & 15, codes >> 4], axis=-1).reshape(*codes.shape[:-1], -1)
    v = np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127.0))
    return v * np.repeat(s, 32, axis=-1)


def random_mx(rng, *shape, lo=118, hi=122):
    """Random codes and scale bytes of an MXFP4 tensor [..., C]."""
    codes = rng.integers(0, 256, shape[:-1] + (shape[-1] // 2,), dtype=np.uint8)
    scales = rng.integers(lo, hi, shape[:-1] + (shape[-1] // 32,), dtype=np.uint8)
    return codes, scales


def product(a, w):
    return mx_decode(*a) @ mx_decode(*w).T


def experts(x_bits, ids, tw, w13, w2):
    """The routed-expert layer; returns (out, magnitude, slots) with, for error
    bounds, the sums of the absolute values of the slots' products and of
    their weighted results."""
    T, H = x_bits.shape
    I = w2[0].shape[-1] * 2
    xh = mx_decode(*mx_encode(x_bits))
    out, mag, slots = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))
    E = w13[0].shape[0]
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if not t.size:
            continue
        gu = xh[t] @ mx_decode(w13[0][e], w13[1][e]).T
        g, u = gu[:, :I], gu[:, I:]
        h = mx_decode(*mx_encode(bf16_round(g / (1.0 + np.exp(-g)) * u)))
        w = mx_decode(w2[0][e], w2[1][e])
        y = (h @ w.T) * tw[t, j, None]
        np.add.at(out, t, y)
        np.add.at(slots, t, np.abs(y))
        np.add.at(mag, t, (np.abs(h) @ np.abs(w).T) * np.abs(tw[t, j, None]))
    return out, mag, slots


# ------------------------------------------------------------------- gate --

def gate(logits, top_k, score="softmax", bias=None, n_group=1, topk_group=1, group_top=1, renormalize=True, scale=1.0):
    """logits float64 [T, E] -> (ids int32, weights float64) by a loop over tokens."""
    T, E = logits.shape
    ids = np.full((T, top_k), -1, np.int32)
    w = np.zeros((T, top_k))
    s_all = np.zeros((T, E))
    for t in range(T):
        l = np.where(np.isnan(logits[t]), -np.inf, np.minimum(logits[t], float(np.finfo(np.float32).max)))
        live = l > -np.inf
        if not live.any():
            continue
        with np.errstate(over="ignore"):
            if score == "softmax":
                e = np.exp(l - l[live].max())
                s = e / e.sum()
            else:
                s = 1.0 / (1.0 + np.exp(-l))
        s_all[t] = s
        plain = bias is None and group_top == 1
        c = l.copy() if plain else s + (0.0 if bias is None else np.asarray(bias, np.float64))
        live &= c > -np.inf
        c = np.where(live, c, -np.inf)
        if topk_group < n_group:
            m = E // n_group
            rank = []
            for g in range(n_group):
                best = sorted((v for v in c[g * m:(g + 1) * m] if v > -np.inf), reverse=True)[:group_top]
                rank.append(sum(best) if best else -np.inf)
            keep = sorted(range(n_group), key=lambda g: (-rank[g], g))[:topk_group]
            for g in range(n_group):
                if g not in keep:
                    c[g * m:(g + 1) * m] = -np.inf
        order = sorted((e for e in range(E) if c[e] > -np.inf), key=lambda e: (-c[e], e))[:top_k]
        ids[t, :len(order)] = order
        if not order:
            continue
        v = s[order]
        if renormalize:
            u = l[order] if score == "softmax" else -np.logaddexp(0.0, -l[order])
            v = np.exp(u - u.max())
            v = v / v.sum()
        w[t, :len(order)] = scale * v
    return ids, w


def gate_weights(logits, ids, score, renormalize, scale):
    """The weights as a function of the logits at fixed ids, for differences."""
    T, E = logits.shape
    w = np.zeros(ids.shape)
    for t in range(T):
        l = logits[t]
        live = l > -np.inf
        j = [i for i, e in enumerate(ids[t]) if 0 <= e < E and live[e]]
        if not j:
            continue
        e = ids[t][j]
        if renormalize:
            u = l[e] if score == "softmax" else -np.logaddexp(0.0, -l[e])
            v = np.exp(u - u.max())
            v = v / v.sum()
        elif score == "softmax":
            v = np.exp(l[e] - l[live].max()) / np.exp(l[live] - l[live].max()).sum()
        else:
            v = 1.0 / (1.0 + np.exp(-l[e]))
        w[t, j] = scale * v
    return w


def gate_gradient(logits, ids, dw, score, renormalize, scale):
    """The gradient by the formulas of the definition, token by token."""
    T, E = logits.shape
    d = np.zeros((T, E))
    w = gate_weights(logits, ids, score, renormalize, scale)
    for t in range(T):
        l = logits[t]
        live = l > -np.inf
        dot = 0.0
        for i, e in enumerate(ids[t]):
            if 0 <= e < E and live[e]:
                dot += w[t, i] * dw[t, i]
        if score == "softmax" and not renormalize and live.any():
            p = np.where(live, np.exp(l - l[live].max()), 0.0)
            d[t] -= dot * p / p.sum()
        for i, e in enumerate(ids[t]):
            if not (0 <= e < E and live[e]):
                continue
            g = w[t, i] * (dw[t, i] - (dot / scale if renormalize else 0.0))
            if score == "sigmoid":
                g /= 1.0 + np.exp(l[e])
            d[t, e] += g
    return d
