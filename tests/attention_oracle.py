"""Attention over a CSR pattern in 64 bits (numpy, row by row), with its
gradients and a bound on the rounding error of an implementation that holds
scores, weights and sums in a type of unit roundoff `u` and rounds its outputs
once to a type of unit roundoff `ut`.

Bound.  A score is a sum of D products, one factor and one sum: it is off by at
most (D + 4) u S, S = scale sum_d |q_d k_d| + |value|.  exp turns that into a
relative error, doubled by the reference (maximum or lse) subtracted from it;
the exponential itself, its argument's scaling and the division add a few u
(16 taken), the sum of L weights L u, and again in the weighted sum of L terms.  A
weight below the type's smallest normal number (2^-126 in 32 bits) may become
zero, whatever its relative error: `eta` more for every weight.
`w`: relative rounding of a weight before it multiplies (tensor cores).
"""
import numpy as np

CODES = {"f64": (2.0 ** -53, 2.0 ** -53, 0.0), "f32": (2.0 ** -24, 2.0 ** -24, 0.0),
         # 16-bit types: sums in 32 bits, weights to 11 bits (bf16) or 20 bits (f16) at least
         "bf16": (2.0 ** -24, 2.0 ** -8, 2.0 ** -11), "f16": (2.0 ** -24, 2.0 ** -11, 2.0 ** -20)}


def attention(rowptr, colind, q, k, v, vals, scale, do=None, code="f64"):
    """q [n, H, D], k and v [m, K, D], vals [nnz] or None, all float64.  Returns a
    dict of results and a dict of error bounds for o, lse and, with do, dq, dk, dv,
    dvals."""
    u, ut, w = CODES[code]
    eta = 2.0 ** -1022 if code == "f64" else 2.0 ** -126
    tiny = {"f16": 2.0 ** -25, "f32": 2.0 ** -120, "bf16": 2.0 ** -120, "f64": 0.0}[code]
    n, H, D = q.shape
    m, K, _ = k.shape
    nnz = colind.shape[0]
    res = {"o": np.zeros((n, H, D)), "lse": np.full((n, H), -np.inf), "dq": np.zeros((n, H, D)),
           "dk": np.zeros((m, K, D)), "dv": np.zeros((m, K, D)), "dvals": np.zeros(nnz)}
    err = {x: np.zeros_like(y) for x, y in res.items()}
    terms = np.bincount(colind, minlength=m) * (H // K)      # of a sum over a column and the heads that share it
    for i in range(n):
        t = np.arange(rowptr[i], rowptr[i + 1])
        if vals is not None:
            t = t[vals[t] != -np.inf]
        if t.size == 0:
            continue
        j = colind[t]
        L = t.size
        for h in range(H):
            g = h // (H // K)
            s = scale * (k[j, g] @ q[i, h]) + (0.0 if vals is None else vals[t])
            S = np.max(abs(scale) * (np.abs(k[j, g]) @ np.abs(q[i, h])) + (0.0 if vals is None else np.abs(vals[t])))
            e = np.exp(s - s.max())
            p = e / e.sum()
            E = u * (2 * (D + 4) * S + 2 * L + 16)
            o = p @ v[j, g]
            oe = (E + w + u * L) * (p @ np.abs(v[j, g]))
            res["o"][i, h] = o
            err["o"][i, h] = oe + ut * (np.abs(o) + oe) + tiny
            res["lse"][i, h] = s.max() + np.log(e.sum())
            err["lse"][i, h] = E + 4 * u * (np.abs(res["lse"][i, h]) + S)
            if do is None:
                continue
            go = do[i, h]
            dp = v[j, g] @ go
            delta = go @ o
            ds = p * (dp - delta)
            dpe = (D + 2) * u * (np.abs(v[j, g]) @ np.abs(go))
            dele = np.abs(go) @ (oe + u * np.abs(o)) + (D + 2) * u * (np.abs(go) @ np.abs(o))
            dse = p * (E * (np.abs(dp) + np.abs(delta)) + dpe + dele) + eta * (np.abs(dp) + np.abs(delta)) + 4 * u * np.abs(ds)
            full = dse + (w + u * (L + 4)) * np.abs(ds)
            res["dq"][i, h] = scale * (ds @ k[j, g])
            err["dq"][i, h] = abs(scale) * (full @ np.abs(k[j, g]))
            res["dvals"][t] += ds
            err["dvals"][t] += dse + 2 * H * u * np.abs(ds)
            np.add.at(res["dk"], (j, g), scale * ds[:, None] * q[i, h])
            np.add.at(err["dk"], (j, g), abs(scale) * (full + u * terms[j] * np.abs(ds))[:, None] * np.abs(q[i, h]))
            np.add.at(res["dv"], (j, g), p[:, None] * go)
            np.add.at(err["dv"], (j, g), ((E + w + u * (terms[j] + 4)) * p + eta)[:, None] * np.abs(go))
    if do is not None:
        for x in ("dq", "dk", "dv"):
            err[x] += ut * (np.abs(res[x]) + err[x]) + tiny
        # dvals has the handle's type: 32 bits unless the tensors have 64
        err["dvals"] += 2.0 ** -24 * np.abs(res["dvals"]) if code != "f64" else 0.0
    return res, err


def within(got, ref, err):
    """The worst error over its bound (at most 1 when every element is within)."""
    d = np.abs(got.astype(np.float64) - ref)
    if not np.isfinite(d).all():
        return np.inf
    return float(np.max(d / np.maximum(err, 1e-300), initial=0.0)) if d.size else 0.0
