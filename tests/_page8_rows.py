"""Attention over the page-scaled formats in 64 bits with a bound for each element, drawn so
tightly that a page left out of a row exceeds it (checked by ``test_page8_bound_host.py``).

A key's weight in the output is p_j (1 + e_j): with dv its page's V scale and w_j = p_j dv,
the kernels hold P'_j = C w_j in fp16, C such that the largest is 2^top or more.
So |e_j| is at most
  2^-11                        P' as fp16, or 2^-25 of it absolutely: 2^(-25-top) max w / w_j,
                               and never more than 1;
  (D/16 + 1) 2^-23 |c| sum|q| dk / sqrt(D)
                               the fp32 accumulation of the scores, codes up to |c| (decode tiles
                               take I8 codes with 128 added: up to 255);
  2^-24 (8 s + 4 log2 dv + 64)  the score's and the exponent's fp32 steps, s the row's largest
                               score in bits; the exponential itself is within 2^-22.
The output is sum p_j (1 + e_j) v_j over the fp32 sum of the p_j (1 + e'_j).  Where the signs of
the values are independent of everything else (they are drawn so), the e_j do not depend on them, and
by Hoeffding's inequality |sum p_j e_j v_j| <= 7 sqrt(sum (p_j e_j v_j)^2) but for one element in 2e10.
``coherent`` takes the plain bound sum p_j e_j |v_j| instead, for values of one sign.
Accumulating the output: one rounding of 2^-23 per 16 keys, of partial sums that the same
inequality bounds; I8 decode tiles count it against the codes' offset of 128, over the at most
64 steps (1024 keys) of a warp.  Its rounding to fp16: 2^-11, or 2^-25 absolutely."""
from __future__ import annotations

import numpy as np

import _page8 as ref

TOP_DECODE, TOP_CHUNK = 7, 6  # log2 of the least largest P'


def attention(fmt, q, codes, scales, row_slots, rows, window=0, missing=(), coherent=False, tops=None, group_rows=24):
    """(o, bound) for packed queries q [total_q, hq, d]; codes, scales = (K, V) planes
    [pages, heads, 32, d] and [pages, heads].  missing[r]: page numbers of row r that count for
    nothing.  Rows of at most group_rows (query, head) rows run on decode tiles."""
    d, hkv = q.shape[2], codes[0].shape[1]
    group = q.shape[1] // hkv
    o, tol, at = np.empty(q.shape), np.empty(q.shape), 0
    for r, (seq, off) in enumerate(rows):
        nq = seq - off
        decode = nq * group <= group_rows
        top = (tops or (TOP_DECODE, TOP_CHUNK))[0 if decode else 1]
        j = np.arange(seq)
        if r < len(missing) and len(missing[r]):
            j = j[~np.isin(j // ref.PAGE, list(missing[r]))]
        s = np.asarray(row_slots[r])[j]
        page, place = s // ref.PAGE, s % ref.PAGE
        dist = np.arange(off, seq)[:, None] - j[None, :]
        seen = (dist >= 0) & ((dist < window) if window else True)
        for h in range(q.shape[1]):
            g = h // group
            dk, dv = (x[page, g].astype(np.float64) for x in scales)
            ck, cv = (x[page, g, place] for x in codes)
            v = cv * dv[:, None]
            qh = q[at:at + nq, h].astype(np.float64)
            x = np.where(seen, (qh @ ck.T) * dk / np.sqrt(d), -np.inf)
            p = np.exp(x - x.max(axis=1, keepdims=True))
            p /= p.sum(axis=1, keepdims=True)
            w = p * dv
            w_max = w.max(axis=1, keepdims=True)
            big = 255.0 if fmt == ref.I8 and decode else (127.0 if fmt == ref.I8 else 448.0)
            score = (d / 16 + 1) * 2.0 ** -23 * big * np.abs(qh).sum(axis=1, keepdims=True) * dk / np.sqrt(d)
            bits = np.abs(np.where(seen, x, 0)).max(axis=1, keepdims=True) * np.log2(np.e)
            log_dv = np.abs(np.log2(dv[dv > 0])).max() if (dv > 0).any() else 0.0
            step = 2.0 ** -22 + 2.0 ** -24 * (8 * bits + 4 * log_dv + 64)
            half = np.minimum(1.0, 2.0 ** -11 + 2.0 ** (-25 - top) * w_max / np.where(w > 0, w, np.inf))
            half = np.where((w > 0) | (dv == 0), half, 1.0)
            pe = p * (half + score + step)
            ps = (p * (score + step)).sum(axis=1, keepdims=True)
            if coherent:
                spread = np.abs(pe) @ np.abs(v)
                sums = p @ np.abs(v)
            else:
                spread = 7 * np.sqrt((pe * pe) @ (v * v))
                sums = 7 * np.sqrt((p * p) @ (v * v))
            out = p @ v
            steps = (min(seq, 1024) if decode else seq) / 16 + 16
            value = steps * 2.0 ** -23 * sums
            if fmt == ref.I8 and decode:
                value += steps * 2.0 ** -23 * 128 * w.sum(axis=1, keepdims=True)
            o[at:at + nq, h] = out
            tol[at:at + nq, h] = 1.01 * (2.0 ** -11 * np.abs(out) + spread + np.abs(out) * ps + value) + 2.0 ** -25
        at += nq
    return o, tol


def off_by(got, want, tol):
    """The largest error as a share of its bound (NaN and infinities count as infinite)."""
    e = np.abs(got.astype(np.float64) - want)
    return float(np.where(np.isfinite(e), e / tol, np.inf).max())
