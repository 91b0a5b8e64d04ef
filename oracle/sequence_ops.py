"""fp64 CPU definitions of the sequence operators (rotary positions, window
attention with sinks, gated linear recurrence) and of their gradients, in
numpy, sharing no code with the CUDA path.

Each function that the kernels are compared with also returns an elementwise
error bound for an evaluation with the kernels' roundings: bf16 results and
bf16 softmax weights (half a step each, 2^-8 relative), everything else in
fp32 (2^-24, with a small constant for the number of operations).
"""
from __future__ import annotations

import math

import numpy as np

HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


# ---------------------------------------------------------------- rotary positions
def rope_frequencies(rot: int, base: float, scaling: dict | None) -> np.ndarray:
    s = scaling or {"kind": "none"}
    if s["kind"] == "base":
        base = base * s["factor"] ** (rot / (rot - 2.0))
    f = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])
    if s["kind"] == "linear":
        f = f / s["factor"]
    if s["kind"] == "ramp":
        r = s["length"] * f / (2 * math.pi)
        keep = np.clip((r - s["low"]) / (s["high"] - s["low"]), 0.0, 1.0)
        f = f * (keep + (1.0 - keep) / s["factor"])
    return f


def rope(x, positions, rot, layout, base=10000.0, scaling=None, inverse=False, dtype="f32"):
    """y and its error bound, x [T, H, d]."""
    x = np.asarray(x, np.float64)
    u = np.asarray(positions, np.float64)[:, None] * rope_frequencies(rot, base, scaling)[None]
    amp = (scaling or {}).get("amplitude", 1.0)
    c, s = amp * np.cos(u)[:, None], amp * np.sin(u)[:, None] * (-1.0 if inverse else 1.0)
    i0 = np.arange(rot // 2) if layout == "half" else np.arange(0, rot, 2)
    i1 = i0 + (rot // 2 if layout == "half" else 1)
    y, tol = x.copy(), np.zeros_like(x)
    a, b = x[..., i0], x[..., i1]
    y[..., i0], y[..., i1] = a * c - b * s, a * s + b * c
    # angle: 2^-25 turns from its fp32 remainder and 2^-25 from 64-bit products of far positions, in radians
    # 3.7e-7; cos, sin, two products and a sum in fp32: 4 2^-24
    size = abs(amp) * (abs(a) + abs(b))
    for i in (i0, i1):
        tol[..., i] = size * (4e-7 + 4 * 2.0 ** -24) + HALF_STEP[dtype] * abs(y[..., i])
    return y, tol


# ---------------------------------------------------------------- window attention
def visible(nq, nk, left, right, sinks):
    p = (nk - nq + np.arange(nq))[:, None]
    u = np.arange(nk)[None]
    return (u <= p + right) & ((u >= p - left) | (u < sinks))


def _spans(cu, rows):
    return [(0, rows)] if cu is None else [(cu[i], cu[i + 1]) for i in range(len(cu) - 1)]


def window_attention(q, k, v, left, right, sinks, cu_q=None, cu_k=None, scale=None, grad_out=None):
    """out, lse and out's error bound; with grad_out also (dq, dk, dv) and theirs.  q [Tq, Hq, d], k, v
    [Tk, Hk, d]; rows outside every sequence are NaN in the results."""
    Tq, Hq, d = q.shape
    Tk, Hk, _ = k.shape
    scale = d ** -0.5 if scale is None else scale
    G = Hq // Hk
    r = {"out": np.full(q.shape, np.nan), "lse": np.full((Hq, Tq), np.nan)}
    r["out_tol"] = np.zeros(q.shape)
    if grad_out is not None:
        for n, like in (("dq", q), ("dk", k), ("dv", k)):
            r[n], r[n + "_tol"] = np.full(like.shape, np.nan), np.zeros(like.shape)
    # weights and dS enter their products with one rounding to bf16; exponentials and their normalisation are
    # good to 2^-10 (a cubic of relative error 7.6e-5 and fp32 arithmetic on exponents of up to some hundreds)
    w_err = 2.0 ** -8 + 2.0 ** -10
    for (q0, q1), (k0, k1) in zip(_spans(cu_q, Tq), _spans(cu_k, Tk)):
        see = visible(q1 - q0, k1 - k0, left, right, sinks)
        for n in ("dk", "dv"):
            if n in r:
                r[n][k0:k1] = 0.0
        for h in range(Hq):
            Q, K, V = (np.asarray(a, np.float64) for a in (q[q0:q1, h], k[k0:k1, h // G], v[k0:k1, h // G]))
            s = np.where(see, scale * Q @ K.T, -np.inf)
            m = s.max(1, initial=-np.inf)
            e = np.exp(s - np.where(np.isfinite(m), m, 0.0)[:, None])
            l = e.sum(1)
            P = e / np.where(l > 0, l, 1.0)[:, None]
            with np.errstate(divide="ignore"):
                r["lse"][h, q0:q1] = np.where(l > 0, np.where(np.isfinite(m), m, 0.0) + np.log(l), -np.inf)
            O = P @ V
            tol = 2.0 ** -8 * abs(O) + w_err * (P @ abs(V))
            r["out"][q0:q1, h], r["out_tol"][q0:q1, h] = O, tol
            if grad_out is None:
                continue
            g = np.asarray(grad_out[q0:q1, h], np.float64)
            dP = g @ V.T
            delta = (g * O).sum(1)
            dS = P * (dP - delta[:, None])
            r["dq"][q0:q1, h] = scale * dS @ K
            r["dk"][k0:k1, h // G] += scale * dS.T @ Q
            r["dv"][k0:k1, h // G] += P.T @ g
            # delta is summed from the rounded output: each element off by at most its bound
            dS_err = w_err * abs(dS) + P * ((abs(g) * tol).sum(1) + 2.0 ** -16 * (abs(g) @ abs(V).T).max(1, initial=0.0))[:, None]
            r["dq_tol"][q0:q1, h] = scale * dS_err @ abs(K) + 2.0 ** -8 * abs(r["dq"][q0:q1, h])
            r["dk_tol"][k0:k1, h // G] += scale * dS_err.T @ abs(Q)
            r["dv_tol"][k0:k1, h // G] += w_err * P.T @ abs(g)
        for n in ("dk", "dv"):
            if n in r:
                r[n + "_tol"][k0:k1] += 2.0 ** -8 * abs(r[n][k0:k1])
    return r


def cache_slot(u, slots, sinks):
    return u if u < slots else sinks + (u - sinks) % (slots - sinks)


def window_decode(q, k_of, v_of, lens, left, sinks, slots, scale=None):
    """One token of each request: k_of(r, u), v_of(r, u) give [Hk, d] of position u.  out and its bound."""
    B, Hq, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(B):
        n = max(int(lens[b]), 0)
        us = [u for u in range(n) if (u >= n - 1 - left or u < sinks) and (u < sinks or n <= slots or u >= n - (slots - sinks))]
        if not us:
            continue
        K = np.stack([np.asarray(k_of(b, u), np.float64) for u in us], 1)
        V = np.stack([np.asarray(v_of(b, u), np.float64) for u in us], 1)
        for h in range(Hq):
            hk = h // (Hq // K.shape[0])
            s = scale * K[hk] @ np.asarray(q[b, h], np.float64)
            p = np.exp(s - s.max())
            p /= p.sum()
            out[b, h] = p @ V[hk]
            tol[b, h] = 2.0 ** -8 * abs(out[b, h]) + (2.0 ** -8 + 2.0 ** -10) * (p @ abs(V[hk]))
    return out, tol


# ---------------------------------------------------------------- gated linear recurrence
def gate(f, form):
    """a, 1 - a, s(a), ds/df."""
    f = np.asarray(f, np.float64)
    with np.errstate(over="ignore"):
        a, rest = 1 / (1 + np.exp(-f)), 1 / (1 + np.exp(f))
    if form == "sum":
        return a, rest, np.ones_like(a), np.zeros_like(a)
    if form == "convex":
        return a, rest, rest, -a * rest
    return a, rest, np.sqrt(rest * (1 + a)), -a * a * np.sqrt(rest / (1 + a))


def gated_scan(f, x, form, reverse=False, cu=None, h0=None, dy=None, dhT=None, dtype="f32"):
    """y, hT and with dy also df, dx, dh0, each with its bound (name + "_tol")."""
    T, D = x.shape
    spans = _spans(cu, T)
    n = len(spans)
    k = 16 * 2.0 ** -24      # a handful of fp32 roundings and two exponentials per step
    r = {"y": np.full((T, D), np.nan), "hT": np.zeros((n, D))}
    r.update({m + "_tol": np.zeros_like(v) for m, v in list(r.items())})
    if dy is not None:
        for m, like in (("df", x), ("dx", x), ("dh0", r["hT"])):
            r[m], r[m + "_tol"] = np.full(like.shape, np.nan), np.zeros(like.shape)
    f, x = np.asarray(f, np.float64), np.asarray(x, np.float64)
    for s, (t0, t1) in enumerate(spans):
        order = range(t1 - 1, t0 - 1, -1) if reverse else range(t0, t1)
        h = np.zeros(D) if h0 is None else np.asarray(h0[s], np.float64)
        size, err = abs(h), np.zeros(D)          # sum of absolute contributions, accumulated error
        keep = []
        for t in order:
            a, rest, g, ds = gate(f[t], form)
            keep.append((t, a, rest, g, ds, h, size, err))
            h = a * h + g * x[t]
            size = a * size + g * abs(x[t])
            err = a * err + k * size
            r["y"][t], r["y_tol"][t] = h, err + HALF_STEP[dtype] * abs(h)
        r["hT"][s], r["hT_tol"][s] = h, err
        if dy is None:
            continue
        lam = np.zeros(D) if dhT is None else np.asarray(dhT[s], np.float64)
        lsize, lerr = abs(lam), np.zeros(D)
        for t, a, rest, g, ds, before, size, err in reversed(keep):
            lam, lsize = lam + dy[t], lsize + abs(dy[t])
            lerr = lerr + k * lsize
            slope = before * a * rest + x[t] * ds
            r["df"][t], r["dx"][t] = lam * slope, lam * g
            span = size * a * rest + abs(x[t] * ds)
            r["df_tol"][t] = (lerr + k * lsize) * span + lsize * err * a * rest + HALF_STEP[dtype] * abs(r["df"][t])
            r["dx_tol"][t] = (lerr + k * lsize) * g + HALF_STEP[dtype] * abs(r["dx"][t])
            lam, lsize, lerr = a * lam, a * lsize, a * (lerr + k * lsize)
        r["dh0"][s], r["dh0_tol"][s] = lam, lerr
    return r
