"""Plain numpy forms of the paged K/V cache operators (fp64 where numbers are computed)."""
from __future__ import annotations

import numpy as np
import torch

BAD_PAGE, NO_PAGE, BAD_ROW = 8, 16, 32


def page_table(lens, page, max_pages, n_pages, pool=None, first=0):
    """(table, held, next, status)."""
    pool = np.arange(n_pages) if pool is None else np.asarray(pool)
    table = np.full((len(lens), max_pages), -1, np.int32)
    held, at, status, full = np.zeros(len(lens), np.int32), first, 0, False
    for b, n in enumerate(lens):
        need = -(-int(n) // page) if n > 0 else 0
        if need > max_pages:
            status |= NO_PAGE
            continue
        if full or at + need > len(pool):
            status |= NO_PAGE if need else 0
            full = full or need > 0
            continue
        for j, pg in enumerate(pool[at:at + need]):
            ok = 0 <= pg < n_pages
            table[b, j] = pg if ok else -1
            status |= 0 if ok else BAD_PAGE
        held[b] = need
        at += need
    return table, held, at, status


def slot_map(table, count, page, n_pages, max_rows, pos=None, first=None):
    """(row_start, row_pos, slot, status); the last two only as long as the rows."""
    B, status = len(table), 0
    row_start, rp, sl = [0], [], []
    for b in range(B):
        k = max(int(count[b]), 0)
        if pos is not None and k > pos.shape[1]:
            k, status = pos.shape[1], status | BAD_ROW
        p = [int(x) for x in pos[b, :k]] if pos is not None else [(int(first[b]) if first is not None else 0) + j
                                                                 for j in range(k)]
        for j, x in enumerate(p):
            if len(rp) == max_rows:
                status |= BAD_ROW
                break
            if pos is not None and j and p[j - 1] >= x:
                status |= BAD_ROW
            pg = table[b, x // page] if 0 <= x and x // page < table.shape[1] else -1
            ok = 0 <= pg < n_pages
            status |= 0 if ok else BAD_PAGE
            rp.append(x)
            sl.append(int(pg) * page + x % page if ok else -1)
        row_start.append(min(row_start[-1] + k, max_rows))
    return np.array(row_start, np.int32), np.array(rp, np.int32), np.array(sl, np.int32), status


def rotate(x, pos, theta):
    """RoPE of x [T][heads][hd] at pos [T]."""
    half = x.shape[-1] // 2
    ang = pos.astype(np.float64)[:, None] * theta ** (-2.0 * np.arange(half) / x.shape[-1])
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    a, b = x[..., :half], x[..., half:]
    return np.concatenate([a * c - b * s, b * c + a * s], -1)


def attention(q, row_start, kv_len, table, k, v, scale):
    """out [T][H][hd], and per element A = sum_j w_j |v_j| and the row's largest sum_d |q_d k_jd| scale (for error
    bounds).  k, v: [n_pages][page][KV][hd] fp64."""
    T, H, hd = q.shape
    n_pages, page, KV, _ = k.shape
    out, A, mag = np.zeros((T, H, hd)), np.zeros((T, H, hd)), np.zeros((T, H))
    for b in range(len(kv_len)):
        lo, hi = int(row_start[b]), int(row_start[b + 1])
        n = min(max(int(kv_len[b]), 0), table.shape[1] * page)
        at = np.arange(n)
        pg = table[b, at // page]
        ok = (pg >= 0) & (pg < n_pages)
        at, pg = at[ok], pg[ok]
        if lo >= hi or not len(at):
            continue
        for h in range(H):
            kk, vv = k[pg, at % page, h // (H // KV)], v[pg, at % page, h // (H // KV)]
            x = q[lo:hi, h] @ kk.T * scale
            w = np.exp(x - x.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            out[lo:hi, h], A[lo:hi, h] = w @ vv, w @ np.abs(vv)
            mag[lo:hi, h] = (np.abs(q[lo:hi, h]) @ np.abs(kk).T * abs(scale)).max(1)
    return out, A, mag


def attention_bound(out, A, mag, dtype, n_keys, hd, p_step):
    """Elementwise error bound of the kernels.  With u = 2^-24: a score is off by at most (hd + 4) u times the
    sum of |q k| scale (products summed in fp32 in any order, the scaling, the fp32 subtraction of the maximum);
    a weight by twice that (numerator and denominator) plus 4 u of the exponential; P is rounded with relative
    step p_step; both sums over keys run in fp32: n u of A each; the result is rounded once to dtype."""
    u = 2.0 ** -24
    half = torch.finfo(dtype).eps / 2
    rel = 2 * ((hd + 4) * u * mag + 4 * u) + p_step + 2 * n_keys * u
    return half * np.abs(out) + rel[..., None] * A * (1 + half) + 1e-30
