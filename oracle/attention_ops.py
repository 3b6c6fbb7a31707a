"""fp64 definitions of the operators of attention layers (include/gdn.h) in numpy, with the error bounds the GPU
tests hold the kernels to.

TEST INFRASTRUCTURE ONLY, like the rest of this package; no code is shared with csrc/.
"""
from __future__ import annotations

import numpy as np

from oracle.layer_ops import HALF_STEP, U32, bound, frequencies, rotary  # noqa: F401

FLUSH = 2.0 ** -126   # fp32's smallest normal value


def norm_rotary(x, w, positions, freq, rot, layout, eps, scale=1.0, dout=None, fast=False):
    """x [B, T, H, d] with integer positions [B, T]; a dict with y and, with dout, dx and dw; ``*_err`` bounds what fp32
    arithmetic adds (the rounding of the result not included).

    Bounds, in units of U32. The sum of squares over d channels: a lane's run of at most d/16 of them, a tree over 32 lanes,
    the products' own roundings: d/16 + 8 relative; half of that in the root, which with the division, eps and the
    reciprocal root's own 2 units comes to kr = d/32 + 8. z = x rstd w: kr + 3 relative. The turn: 8 of |z1| + |z2| for the
    fp32 angle and products, 16 where cos and sin are the hardware's (`fast`; see the rotary tests).
    """
    x = np.asarray(x, np.float64)
    d = x.shape[-1]
    w = np.ones(d) if w is None else np.asarray(w, np.float64)
    kr, kt = d / 32.0 + 8.0, 16.0 if fast else 8.0
    rstd = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * rstd
    z = xh * w
    half = rot // 2
    i1 = np.arange(half) if layout == "half" else 2 * np.arange(half)
    i2 = i1 + half if layout == "half" else i1 + 1

    def pair_size(v):
        m = np.abs(v).copy()
        m[..., i1] = m[..., i2] = (np.abs(v[..., i1]) + np.abs(v[..., i2])) * abs(scale)
        return m

    r = {"y": rotary(z, positions, freq, rot, layout, scale=scale), "y_err": U32 * (kr + 3 + kt) * pair_size(z)}
    if dout is None:
        return r
    g = np.asarray(dout, np.float64)
    dz, edz = rotary(g, positions, freq, rot, layout, inverse=True, scale=scale), U32 * kt * pair_size(g)
    t, et = dz * w, np.abs(w) * (edz + U32 * np.abs(dz))
    m = (t * xh).mean(-1, keepdims=True)
    em = (et * np.abs(xh)).mean(-1, keepdims=True) + U32 * (kr + d / 16.0 + 12) * np.abs(t * xh).mean(-1, keepdims=True)
    r["dx"] = rstd * (t - xh * m)
    r["dx_err"] = rstd * (et + np.abs(xh) * em + U32 * (2 * kr + 6) * (np.abs(t) + np.abs(xh * m)))
    terms, ez = dz * xh, edz * np.abs(xh) + U32 * (kr + 3) * np.abs(dz * xh)
    rows = terms[..., 0].size
    axes = tuple(range(terms.ndim - 1))
    # fp32 sums: at most one rounding per addend, of a partial sum no larger than the sum of the absolute values
    r["dw"], r["dw_err"] = terms.sum(axes), ez.sum(axes) + U32 * (rows + 32) * np.abs(terms).sum(axes)
    return r


def visible(Lq, Lk, window, sinks):
    """[Lq, Lk] truth values: which keys each query sees."""
    p = (Lk - Lq + np.arange(Lq))[:, None]
    j = np.arange(Lk)[None]
    return (j <= p) & ((p - j < window) | (j < sinks))


def window_attention(q, k, v, window, sinks, scale, dtype, dout=None):
    """One sequence: q [Lq, Hq, d], k, v [Lk, Hk, d] in fp64 holding values of `dtype`. A dict with out [Lq, Hq, d], lse
    [Hq, Lq] and, with dout, dq, dk, dv; each with a bound ``*_err`` on what the kernels may add before they round the
    result once.

    Bounds. A score is a sum of d products that are exact (16 bits) or rounded, in fp32, in any order, an addition
    rounding or cutting off: es = (2d + 8) U32 scale sum |q||k|. exp's argument and value: rp = es + U32 (4 (|s| + the
    row's largest |s|) + 8) relative to P. For 16-bit types the weights are rounded to the type before the product with v:
    relative eps = half a step, and absolutely, of weights whose largest is at least 1 (so that the sum l >= 1), `least`, half of
    the type's smallest step, for fp16 in units of 2^-6, in which they are held. l itself is added up in fp32 unrounded: n U32.
    The product with v adds 2n U32.
    Backward: P = exp(s - lse) with lse's own error; delta = sum dO O takes O's error and rounding; dS = scale P (dP - delta) is
    rounded to the type, as P is; the sums over n keys (or queries and heads) add 2n U32. fp16 holds P in units of 2^-12 and
    P (dP - delta) in units of 2^-12 / f, with a power of two f >= 2 / b, where b = 2 max |dO| max |v| (2-norms of rows, over the
    sequence and the heads that share keys) bounds |dP - delta|: absolutely least 2^-12, and least scale b 2^-13.
    The hardware's exponential counts a result below 2^-126, the smallest normal fp32, as 0 (ex2.approx.ftz): a weight, whose
    row's largest is at least 1, and a P are off by up to 2^-126 more.
    """
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    Lq, Hq, d = q.shape
    Lk, Hk, _ = k.shape
    G = Hq // Hk
    eps, least = HALF_STEP[dtype] if dtype != "fp32" else (0.0, 0.0)
    step = HALF_STEP[dtype][0]
    half = dtype == "fp16"
    least_w, least_p = (least * 2.0 ** -6, least * 2.0 ** -12) if half else (least, least)
    see = visible(Lq, Lk, window, sinks)
    any_seen = see.any(1)
    r = {"out": np.zeros((Lq, Hq, d)), "out_err": np.zeros((Lq, Hq, d)), "lse": np.full((Hq, Lq), -np.inf), "lse_err": np.zeros((Hq, Lq))}
    if dout is not None:
        dout = np.asarray(dout, np.float64)
        for n, x in (("dq", q), ("dk", k), ("dv", v)):
            r[n], r[n + "_err"] = np.zeros(x.shape), np.zeros(x.shape)
    if Lq == 0 or Lk == 0:
        return r
    n_row = see.sum(1)[:, None]
    n_col = see.sum(0)[:, None] * G
    for h in range(Hq):
        Q, K, V = q[:, h], k[:, h // G], v[:, h // G]
        aQ, aK, aV = np.abs(Q), np.abs(K), np.abs(V)
        s = np.where(see, scale * (Q @ K.T), -np.inf)
        es = U32 * (2 * d + 8) * scale * (aQ @ aK.T)
        top = np.where(any_seen, np.where(see, s, -np.inf).max(1), 0.0)[:, None]
        big = np.abs(np.where(see, s, 0.0)).max(1)[:, None]
        w = np.where(see, np.exp(np.where(see, s, 0.0) - top), 0.0)
        l = np.where(any_seen, w.sum(1), 1.0)[:, None]
        P = w / l
        rp = np.where(see, es + U32 * (4 * (np.abs(np.where(see, s, 0.0)) + big) + 8), 0.0)
        mean_rp = (P * rp).sum(1)[:, None]
        O = P @ V
        eO = (P * (eps + rp)) @ aV + (mean_rp + U32 * (3 * n_row + 16)) * (P @ aV) + (least_w + FLUSH) * (see @ aV)
        lse = np.where(any_seen, top[:, 0] + np.log(l[:, 0]), -np.inf)
        elog = mean_rp[:, 0] + U32 * (n_row[:, 0] + 8 + 4 * np.abs(np.where(any_seen, lse, 0.0)) + 2 * big[:, 0])
        r["out"][:, h], r["out_err"][:, h] = O, eO
        r["lse"][h], r["lse_err"][h] = lse, elog
        if dout is None:
            continue
        g = dout[:, h]
        ag = np.abs(g)
        delta = (g * O).sum(1)[:, None]
        edelta = (ag * (eO * (1 + step) + step * np.abs(O))).sum(1)[:, None] + U32 * (d + 8) * (ag * np.abs(O)).sum(1)[:, None]
        dP, edP = g @ V.T, U32 * (2 * d + 8) * (ag @ aV.T)
        rP = rp + elog[:, None] + U32 * (4 * np.abs(np.where(any_seen, lse, 0.0))[:, None] + 8)
        dS = scale * P * (dP - delta)
        edS = scale * FLUSH * see * (np.abs(dP - delta) + edP + edelta) + scale * P * (rP * np.abs(dP - delta) + edP + edelta + 4 * U32 * (np.abs(dP) + np.abs(delta)))
        least_s = least
        if half:
            heads = slice(h // G * G, h // G * G + G)
            least_s = least * scale * 2 * np.sqrt((dout[:, heads] ** 2).sum(-1).max() * (V ** 2).sum(-1).max()) * 2.0 ** -13
        edS = edS + eps * (np.abs(dS) + edS) + least_s * see
        eP = P * (rP + eps * (1 + rP)) + (least_p + FLUSH) * see
        r["dq"][:, h] = dS @ K
        r["dq_err"][:, h] = edS @ aK + 2 * U32 * n_row * (np.abs(dS) @ aK)
        r["dk"][:, h // G] += dS.T @ Q
        r["dk_err"][:, h // G] += edS.T @ aQ + 2 * U32 * n_col * (np.abs(dS).T @ aQ)
        r["dv"][:, h // G] += P.T @ g
        r["dv_err"][:, h // G] += eP.T @ ag + 2 * U32 * n_col * (P.T @ ag)
    return r


def slot_of(p, sinks, slots):
    return p if p < sinks else sinks + (p - sinks) % (slots - sinks)


def cache_write(cache, new, lengths, sinks):
    """cache [N, Hk, slots, d], new a list of [T_n, Hk, d]: token by token, in order."""
    out = np.array(cache)
    for n, x in enumerate(new):
        if lengths[n] < 0:
            continue
        for t in range(x.shape[0]):
            out[n, :, slot_of(int(lengths[n]) + t, sinks, out.shape[2])] = x[t]
    return out


def step(q, kc, vc, lengths, window, sinks, scale, dtype):
    """q [N, Hq, d] over caches that hold the new token already: (out, out_err) [N, Hq, d]."""
    N, Hq, d = q.shape
    out, err = np.zeros(q.shape), np.zeros(q.shape)
    for n in range(N):
        t = int(lengths[n])
        if t < 0:
            continue
        pos = [p for p in range(t + 1) if t - p < window or p < sinks] if t < 4096 else \
            list(range(min(sinks, t - window + 1))) + list(range(max(0, t - window + 1), t + 1))
        idx = [slot_of(p, sinks, kc.shape[2]) for p in pos]
        K, V = kc[n][:, idx].transpose(1, 0, 2), vc[n][:, idx].transpose(1, 0, 2)
        r = window_attention(q[n][None], K, V, len(idx), 0, scale, dtype)
        out[n], err[n] = r["out"][0], r["out_err"][0]
    return out, err
