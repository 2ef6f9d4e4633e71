"""Attention inside the cells of a partition, in fp64 numpy: window attention with a learned
relative position bias by buckets, differential attention, rows in 8 bits.

Test infrastructure; shares no code with the CUDA path.  Written cell by cell from the
formulas, gradients by the chain rule.  Beside each result stands a bound on how far an
evaluation may be off whose products and sums are fp32 and that rounds the softmax weights
and dS to storage with unit roundoff `u` before the second products (bf16: 2^-8; fp32: 0) and
the result to storage with roundoff `u_out`:

  * a score is off by at most e_s = (d + 4) 2^-24 S with S = the largest sum of |terms| of a
    score of the row; a weight p by a relative e_p = 2 e_s + 2^-20 (two exponentials' worth of
    e_s from the score and the normaliser; 2^-22 for ex2.approx, the sum and the division);
  * dP by (d + 4) 2^-24 A, A = sum |dout| |v|; D = sum p dP by e_p + that, summed;
  * a sum of terms t_j with relative errors e: sum |t_j| (e + u) + u_out |result|, and
    n 2^-24 sum |t_j| for the n additions.
"""
from __future__ import annotations

import numpy as np

EPS = 2.0 ** -24


def offset_number(ci, cj, m):
    """Number of the offsets ci - cj (window edge m): [ni, nj]."""
    e = 2 * m - 1
    o = ci[:, None, :] - cj[None, :, :] + (m - 1)
    return (o[..., 0] * e + o[..., 1]) * e + o[..., 2]


def _softmax(s):
    """Rows of minus infinity give zeros."""
    mx = s.max(-1, keepdims=True)
    mx = np.where(np.isneginf(mx), 0.0, mx)
    x = np.exp(s - mx)
    l = x.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        return x / np.where(l == 0, 1.0, l), (mx + np.log(l))[..., 0]


def cells(ids, count):
    """Tokens of each cell, ascending."""
    return [np.nonzero(np.asarray(ids) == c)[0] for c in range(count)]


def window(ids, count, q, k, v, dout, scale, coords=None, m=0, table=None, bucket=None, u=0.0, u_out=0.0):
    """Values and bounds: dict name -> (value, bound) for out, lse, dq, dk, dv, dbias."""
    q, k, v, dout = (np.asarray(x, np.float64) for x in (q, k, v, dout))
    n, hq, d = q.shape
    hkv = k.shape[1]
    g = hq // hkv
    z = {x: [np.zeros_like(y), np.zeros_like(y)] for x, y in
         (("out", q), ("dq", q), ("dk", k), ("dv", v))}
    z["lse"] = [np.full((n, hq), -np.inf), np.zeros((n, hq))]
    if table is not None:
        table = np.asarray(table, np.float64)
        table = np.where(table <= -1e38, -np.inf, table)  # lowest values bar as minus infinity does
        nb = table.shape[1]
        z["dbias"] = [np.zeros_like(table), np.zeros_like(table)]
    fd = (d + 4) * EPS
    for tok in cells(ids, count):
        if not len(tok):
            continue
        if table is not None:
            off = offset_number(np.asarray(coords)[tok].astype(np.int64) % m, np.asarray(coords)[tok].astype(np.int64) % m, m)
            b = off if bucket is None else np.asarray(bucket)[off]
            has = (b >= 0) & (b < nb)
            b = np.where(has, b, 0)
        for h in range(hq):
            qi, kj, vj, do = q[tok, h], k[tok, h // g], v[tok, h // g], dout[tok, h]
            s = scale * qi @ kj.T
            sa = scale * np.abs(qi) @ np.abs(kj).T
            if table is not None:
                t = np.where(has, table[h][b], 0.0)
                s = s + t
                sa = sa + np.where(np.isfinite(t), np.abs(t), 0.0)
            p, lse = _softmax(s)
            es = fd * sa.max(-1, keepdims=True)
            ep = 2 * es + 2.0 ** -20
            z["lse"][0][tok, h] = lse
            z["lse"][1][tok, h] = es[:, 0] + 2.0 ** -20 + 4 * EPS * np.abs(np.where(np.isfinite(lse), lse, 0))
            add = len(tok) * EPS
            o = p @ vj
            z["out"][0][tok, h] = o
            z["out"][1][tok, h] = (p * (ep + u + add)) @ np.abs(vj) + u_out * np.abs(o)
            dp, A = do @ vj.T, np.abs(do) @ np.abs(vj).T
            D = (p * dp).sum(-1, keepdims=True)
            eD = (p * (np.abs(dp) * (ep + add) + fd * A)).sum(-1, keepdims=True)
            ds = p * (dp - D)
            eds = p * (np.abs(dp - D) * (ep + 4 * EPS) + fd * A + eD)
            z["dq"][0][tok, h] += scale * ds @ kj
            z["dq"][1][tok, h] += scale * (eds + np.abs(ds) * (u + add)) @ np.abs(kj)
            z["dk"][0][tok, h // g] += scale * ds.T @ qi
            addk = g * add
            z["dk"][1][tok, h // g] += scale * (eds + np.abs(ds) * (u + addk)).T @ np.abs(qi)
            z["dv"][0][tok, h // g] += p.T @ do
            z["dv"][1][tok, h // g] += (p * (ep + u + addk)).T @ np.abs(do)
            if table is not None:
                np.add.at(z["dbias"][0][h], b[has], ds[has])
                np.add.at(z["dbias"][1][h], b[has], (eds + np.abs(ds) * n * EPS)[has])
    for x in ("dq", "dk", "dv"):
        z[x][1] += u_out * np.abs(z[x][0])
    return {x: tuple(y) for x, y in z.items()}


def diff_lambda(lam, lam_init):
    lam = np.asarray(lam, np.float64)
    e1, e2 = np.exp((lam[0] * lam[1]).sum(-1)), np.exp((lam[2] * lam[3]).sum(-1))
    return e1, e2, e1 - e2 + lam_init


def diff(ids, count, q, k, v, dout, scale, lam, lam_init, u=0.0, u_out=0.0):
    """Values and bounds: dict name -> (value, bound) for out, dq, dk, dv, dlam."""
    q, k, v, dout, lam = (np.asarray(x, np.float64) for x in (q, k, v, dout, lam))
    n, hq, d = q.shape
    hkv = k.shape[1]
    g = hq // hkv
    z = {x: [np.zeros_like(y), np.zeros_like(y)] for x, y in
         (("out", q), ("dq", q), ("dk", k), ("dv", v), ("dlam", lam))}
    e1, e2, lams = diff_lambda(lam, lam_init)
    fd = (2 * d + 4) * EPS
    # lambda itself: two dot products, two exponentials (2 ulp each), two additions
    elam = (d + 8) * EPS * ((np.abs(lam[0] * lam[1]).sum(-1) + 1) * e1 + (np.abs(lam[2] * lam[3]).sum(-1) + 1) * e2
                            + abs(lam_init))
    dl, edl = np.zeros(hq // 2), np.zeros(hq // 2)
    for tok in cells(ids, count):
        if not len(tok):
            continue
        add = len(tok) * EPS
        for h in range(hq // 2):
            hk = h // g
            vj = np.concatenate([v[tok, 2 * hk], v[tok, 2 * hk + 1]], 1)
            do = np.concatenate([dout[tok, 2 * h], dout[tok, 2 * h + 1]], 1)
            L, eL = lams[h], elam[h]
            dp, A = do @ vj.T, np.abs(do) @ np.abs(vj).T
            maps = []
            for x in (0, 1):
                qi, kj = q[tok, 2 * h + x], k[tok, 2 * hk + x]
                p, _ = _softmax(scale * qi @ kj.T)
                ep = 2 * fd * (scale * np.abs(qi) @ np.abs(kj).T).max(-1, keepdims=True) + 2.0 ** -20
                maps.append((p, ep))
                w, ew = (1.0, 0.0) if x == 0 else (-L, eL)
                D = (p * dp).sum(-1, keepdims=True)
                eD = (p * (np.abs(dp) * (ep + add) + fd * A)).sum(-1, keepdims=True)
                ds = w * p * (dp - D)
                eds = abs(w) * p * (np.abs(dp - D) * (ep + 4 * EPS) + fd * A + eD) + ew * p * np.abs(dp - D)
                z["dq"][0][tok, 2 * h + x] += scale * ds @ kj
                z["dq"][1][tok, 2 * h + x] += scale * (eds + np.abs(ds) * (u + add)) @ np.abs(kj)
                z["dk"][0][tok, 2 * hk + x] += scale * ds.T @ qi
                z["dk"][1][tok, 2 * hk + x] += scale * (eds + np.abs(ds) * (u + g * add)).T @ np.abs(qi)
                if x:
                    dl[h] -= D.sum()
                    edl[h] += eD.sum()
            (p1, ep1), (p2, ep2) = maps
            w = p1 - L * p2
            ew = p1 * ep1 + abs(L) * p2 * (ep2 + 2 * EPS) + eL * p2
            o = w @ vj
            # the forward rounds each map on its own: u (p1 + |lambda| p2), not u |p1 - lambda p2|
            eo = (ew + (p1 + abs(L) * p2) * (u + add)) @ np.abs(vj)
            gv = w.T @ do
            ev = (ew + np.abs(w) * (u + g * add)).T @ np.abs(do)
            for x in (0, 1):
                c = slice(x * d, x * d + d)
                z["out"][0][tok, 2 * h + x] = o[:, c]
                z["out"][1][tok, 2 * h + x] = eo[:, c] + u_out * np.abs(o[:, c])
                z["dv"][0][tok, 2 * hk + x] += gv[:, c]
                z["dv"][1][tok, 2 * hk + x] += ev[:, c]
    for x in ("dq", "dk", "dv"):
        z[x][1] += u_out * np.abs(z[x][0])
    for i, j, e, sign in ((0, 1, e1, 1.0), (1, 0, e1, 1.0), (2, 3, e2, -1.0), (3, 2, e2, -1.0)):
        z["dlam"][0][i] = sign * (dl * e)[:, None] * lam[j]
        arg = (np.abs(lam[i] * lam[j]).sum(-1) + 1) * (d + 8) * EPS
        z["dlam"][1][i] = ((edl + np.abs(dl) * (arg + 8 * EPS)) * e)[:, None] * np.abs(lam[j])
    return {x: tuple(y) for x, y in z.items()}


def act8(x):
    """(codes, scale) of rows x [..., d] held as float: scale the smallest power of two, at
    least 2^-126, with |x| <= 127 scale (1 for zeros, NaN for rows that are not finite); codes the nearest whole numbers whose
    value is finite in fp32."""
    x = np.asarray(x, np.float64)
    codes, scale = np.zeros(x.shape, np.int8), np.empty(x.shape[:-1])
    for i in np.ndindex(*x.shape[:-1]):
        top = np.abs(x[i]).max()
        if not np.isfinite(top):
            scale[i] = np.nan
            continue
        s = 2.0 ** -126 if top else 1.0
        while top > 127 * s:
            s *= 2
        scale[i] = s
        most = 63 if s == 2.0 ** 122 else 127  # 64 * 2^122 is no fp32 number
        codes[i] = np.clip(np.rint(x[i] / s), -most, most).astype(np.int8)
    return codes, scale
