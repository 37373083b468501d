"""fp64 CPU oracle for the packed append, the packed prompt attention and the
verification of drafted tokens.

TEST INFRASTRUCTURE ONLY, like ``mla_oracle``; it shares no code with the CUDA
library and never imports it.
"""

from __future__ import annotations

import numpy as np

from . import cache_write as cw


def packed_positions(cu, seq_lens):
    """(rows, sequence, position) of every token of a packed batch."""
    rows, seq, pos = [], [], []
    for b in range(len(seq_lens)):
        n = int(cu[b + 1]) - int(cu[b])
        for i in range(n):
            rows.append(int(cu[b]) + i)
            seq.append(b)
            pos.append(int(seq_lens[b]) - n + i)
    return np.array(rows, int), np.array(seq, int), np.array(pos, int)


def append_rows(c, k_pe, cu, seq_lens, rope_base=10000.0):
    """Exact cache rows [tokens][576] of a packed batch, with their rows and positions."""
    rows, seq, pos = packed_positions(cu, seq_lens)
    if rows.size == 0:
        return rows, seq, pos, np.zeros((0, 576))
    return rows, seq, pos, np.concatenate([c[rows], cw.rope(k_pe[rows], pos, rope_base)], axis=1)


def attend_packed(q, k, v, cu, scale, causal):
    """Per sequence and head: (o, lse, sum_j p_j |v_j|, max_j sum_d |q_d k_jd| scale),
    for q [n][H][d], k [n][H_kv][d], v [n][H_kv][dv].  Rows of no sequence are NaN."""
    n, H, _ = q.shape
    share = H // k.shape[1]
    o = np.full((n, H, v.shape[2]), np.nan)
    lse = np.full((n, H), np.nan)
    mass, size = np.full_like(o, np.nan), np.full_like(lse, np.nan)
    for b in range(len(cu) - 1):
        lo, hi = int(cu[b]), int(cu[b + 1])
        for h in range(H):
            kk, vv = k[lo:hi, h // share], v[lo:hi, h // share]
            for i in range(lo, hi):
                m = i + 1 - lo if causal else hi - lo
                s = scale * (kk[:m] @ q[i, h])
                top = s.max()
                p = np.exp(s - top)
                l = p.sum()
                o[i, h] = (p / l) @ vv[:m]
                lse[i, h] = top + np.log(l)
                mass[i, h] = (p / l) @ np.abs(vv[:m])
                size[i, h] = scale * (np.abs(kk[:m]) @ np.abs(q[i, h])).max()
    return o, lse, mass, size


def verify_draft(p, q, draft, num, u_accept, u_sample, seq_lens):
    """(tokens, accepted, new_lens); p [B][S + 1][V], q [B][S][V] or None."""
    B, rows, V = p.shape
    draft, u_accept = np.asarray(draft), np.asarray(u_accept)
    tokens = np.full((B, rows), -1, np.int64)
    accepted, new_lens = np.zeros(B, np.int64), np.array(seq_lens, np.int64)
    for b in range(B):
        n, a = int(num[b]), 0
        while a < n:
            x = int(draft[b, a])
            qx = 1.0 if q is None else float(q[b, a, x])
            if not float(u_accept[b, a]) * qx < float(p[b, a, x]):
                break
            tokens[b, a] = x
            a += 1
        target = np.maximum(p[b, a].astype(np.float64), 0.0)
        w = target.copy()
        if a < n:
            if q is None:
                w[int(draft[b, a])] -= 1.0
            else:
                with np.errstate(invalid="ignore"):
                    w = w - np.maximum(q[b, a].astype(np.float64), 0.0)
        w = np.where(w > 0, w, 0.0)
        if a < n and not w.sum() > 0:
            w = np.where(target > 0, target, 0.0)
        sums = np.cumsum(w)
        if sums[-1] > 0 and np.isfinite(sums[-1]) and not np.isposinf(target).any():
            tokens[b, a] = int(np.searchsorted(sums, float(u_sample[b]) * sums[-1], side="right"))
        accepted[b], new_lens[b] = a, new_lens[b] - (n - a)
    return tokens, accepted, new_lens
