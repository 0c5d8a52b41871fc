"""Float64 reference of the windowed attention, the position rotation and the paged cache,
with bounds on the error that bf16 tensor-core arithmetic may make.

Query i of a sequence with Lq queries and Lk keys stands at p = i + Lk - Lq and sees key j
iff j <= p and (j > p - window or j < sinks).  Query head h reads key/value head
h // (H // H_kv).  Everything is computed densely, one sequence and head at a time.

Error bounds (elementwise).  u = 2^-8 is half a bf16 step, relative.  The kernels hold
scores, exponentials, sums and accumulators in fp32; what they round to bf16 is P, dS, the
outputs and (between the passes) O.  With e_s the error of a score -- an fp32 sum of d exact
products, (d + 8) 2^-24 times the sum of their magnitudes, and 2^-20 for the exponential --
and A = sum_j P_j |v_j|:
  out   u |out| + (u + 4 e_s) A
  lse   e_s + 2^-20 (1 + |lse|)
  dv_j  u |dv| + sum_i (u + 4 e_s) P_ij |dO_i|
  D_i   sum_c |dO_c| (err out_c) + 2^-20 sum_c |dO_c out_c|
  dS_ij P_ij (err D_i + 2^-20 sum |dO_c v_c|) + (u + 4 e_s) |dS_ij|
  dq_i  u |dq| + scale sum_j err dS_ij |k_j|,  dk_j likewise with |q_i|
The last factors carry 2^-18 more for the fp32 accumulation of these sums.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -8
E = 2.0 ** -20


def f64(x):
    if hasattr(x, "detach"):
        x = x.detach().cpu()
        x = x.double().numpy() if x.is_floating_point() else x.numpy()
    return np.asarray(x)


def visible(lq, lk, window, sinks):
    p = np.arange(lq)[:, None] + (lk - lq)
    j = np.arange(lk)[None, :]
    return (j <= p) & ((j > p - window) | (j < sinks))


def _softmax(s, see):
    s = np.where(see, s, -np.inf)
    m = s.max(axis=-1, initial=-np.inf, keepdims=True)
    m = np.where(np.isneginf(m), 0.0, m)
    e = np.exp(s - m)
    total = e.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (m + np.log(total))[..., 0]
    return e / np.where(total > 0, total, 1.0), lse


def window_attention(q, k, v, q_off, kv_off, window, sinks, scale, dout=None):
    """{name: (value, bound)} for out, lse and, with dout, dq, dk, dv."""
    q, k, v, q_off, kv_off = (f64(x) for x in (q, k, v, q_off, kv_off))
    dout = None if dout is None else f64(dout)
    (Tq, H, d), G = q.shape, k.shape[1]
    group = H // G
    val = {"out": np.zeros(q.shape), "lse": np.full((H, Tq), -np.inf)}
    if dout is not None:
        val.update(dq=np.zeros(q.shape), dk=np.zeros(k.shape), dv=np.zeros(v.shape))
    err = {n: np.zeros(x.shape) for n, x in val.items()}
    for b in range(len(q_off) - 1):
        qs, ks = slice(q_off[b], q_off[b + 1]), slice(kv_off[b], kv_off[b + 1])
        lq, lk = qs.stop - qs.start, ks.stop - ks.start
        if lq == 0 or lk == 0:
            continue
        see = visible(lq, lk, window, sinks)
        for h in range(H):
            g = h // group
            Q, K, V = q[qs, h], k[ks, g], v[ks, g]
            # what no query sees plays no part, whatever it holds
            seen = see.any(0)
            K, V = np.where(seen[:, None], K, 0.0), np.where(seen[:, None], V, 0.0)
            P, lse = _softmax(scale * (Q @ K.T), see)
            es = ((d + 8) * 2.0 ** -24 * scale * (np.abs(Q) @ np.abs(K).T) * see).max(-1, keepdims=True) + E
            O, A = P @ V, P @ np.abs(V)
            eo = U * np.abs(O) + (U + 4 * es) * A
            val["out"][qs, h], err["out"][qs, h] = O, eo
            val["lse"][h, qs] = lse
            err["lse"][h, qs] = es[:, 0] + E * (1 + np.abs(np.where(np.isneginf(lse), 0, lse)))
            if dout is None:
                continue
            dO = dout[qs, h]
            dP = dO @ V.T
            D = (dO * O).sum(-1, keepdims=True)
            eD = (np.abs(dO) * eo).sum(-1, keepdims=True) + E * (np.abs(dO * O)).sum(-1, keepdims=True)
            dS = P * (dP - D)
            eS = P * (eD + E * (np.abs(dO) @ np.abs(V).T)) + (U + 4 * es) * np.abs(dS)
            acc = 2.0 ** -18
            val["dq"][qs, h] = scale * dS @ K
            err["dq"][qs, h] = U * np.abs(scale * dS @ K) + scale * (eS + acc * np.abs(dS)) @ np.abs(K)
            val["dk"][ks, g] += scale * dS.T @ Q
            err["dk"][ks, g] += scale * (eS + acc * np.abs(dS)).T @ np.abs(Q)
            val["dv"][ks, g] += P.T @ dO
            err["dv"][ks, g] += ((U + 4 * es + acc) * P).T @ np.abs(dO)
    for n in ("dk", "dv"):
        if n in val:
            err[n] += U * np.abs(val[n])
    return {n: (val[n], err[n]) for n in val}


def rotate(x, positions, frequencies, interleaved=False):
    """(value, bound): rows x [T, heads, d] rotated by their positions; the rest of each head
    beyond 2 * len(frequencies) elements is unchanged.  Bound: one bf16 rounding, plus angles
    good to 2^-31 turns with 2^-22 for sine, cosine and the products."""
    x, f = f64(x), f64(frequencies)
    r = 2 * len(f)
    t = np.asarray(positions, dtype=np.float64)[:, None, None] * f
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
    new_a, new_b = a * np.cos(t) - b * np.sin(t), b * np.cos(t) + a * np.sin(t)
    size = (np.abs(a) + np.abs(b)) * (2.0 ** -22 + 2.0 ** -28)
    val, err = x.copy(), np.zeros(x.shape)
    for at, n in ((0, new_a), (1, new_b)):
        sl = (..., slice(at, r, 2)) if interleaved else (..., slice(at * (r // 2), (at + 1) * (r // 2)))
        val[sl], err[sl] = n, U * np.abs(n) + size
    return val, err


def cache_rows(cache, page_table, b, positions):
    """Rows [len(positions), H_kv, d] of sequence b in a paged cache."""
    cache, page_table = f64(cache), f64(page_table)
    page = cache.shape[2]
    positions = np.asarray(positions, dtype=np.int64)
    return cache[page_table[b][positions // page], :, positions % page]


def cache_attention(q, k_cache, v_cache, page_table, lengths, window, sinks, scale):
    """{name: (value, bound)} for out [B, H, d] and lse [H, B]."""
    q, lengths = f64(q), f64(lengths)
    B, H, d = q.shape
    val = {"out": np.zeros(q.shape), "lse": np.full((H, B), -np.inf)}
    err = {n: np.zeros(x.shape) for n, x in val.items()}
    for b in range(B):
        L = int(lengths[b])
        j = np.arange(L)
        j = j[(j >= L - window) | (j < sinks)]
        if not len(j):
            continue
        K, V = (cache_rows(c, page_table, b, j) for c in (k_cache, v_cache))
        r = window_attention(q[b][None], K, V, [0, 1], [0, len(j)], len(j), 0, scale)
        for n in val:
            for into, x in ((val, r[n][0]), (err, r[n][1])):
                if n == "out":
                    into[n][b] = x[0]
                else:
                    into[n][:, b] = x[:, 0]
    return {n: (val[n], err[n]) for n in val}
