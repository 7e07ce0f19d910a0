"""Float64 reference of attention with shaped scores (soft cap, distance bias, visible
ranges), straight from its definition, on the CPU.

TEST INFRASTRUCTURE ONLY.  Tensors are torch CPU tensors; pools are given in their stored
type and results are float64.  Decode, and decode with shared prefixes, are the same thing
with the last q_len tokens of each sequence as its rows.
"""
import math

import torch

from oracle import page_ops as ref


def score(s, softcap, slope, far):
    """A shaped score, in Python floats."""
    if softcap:
        s = softcap * math.tanh(s / softcap)
    return s - slope * abs(far)


def attend(q, k_pool, v_pool, k_scale, v_scale, cu, table, lens, scale, causal=True, window=0,
           softcap=0.0, slopes=None, visible=None):
    """({row: out [Hq, D]}, {row: sum_t p_t |v_t| / sum_t p_t}), float64."""
    hq, hkv, bs = q.shape[1], k_pool.shape[2], k_pool.shape[1]
    group, d = hq // hkv, q.shape[2]
    out, size = {}, {}
    for b in range(len(lens)):
        L = int(lens[b])
        rows = ref.rows_of(cu, lens, b)
        if not rows:
            continue
        zero = torch.zeros(hkv, d, dtype=torch.float64)
        at = [ref.place(table, bs, b, t) if int(table[b][t // bs]) >= 0 else None
              for t in range(L)]
        k, v = [torch.stack([ref.values(p, s, *a) if a else zero for a in at] or [zero])[:L]
                for p, s in ((k_pool, k_scale), (v_pool, v_scale))]
        for row, pos in rows:
            lo, hi = 0, L
            if causal:
                hi = pos + 1
                lo = max(0, pos - window + 1) if window else 0
            if visible is not None:
                lo, hi = max(lo, int(visible[row][0])), min(hi, int(visible[row][1]))
            if hi <= lo:
                out[row] = torch.zeros(hq, d, dtype=torch.float64)
                size[row] = out[row]
                continue
            qr = q[row].double().view(hkv, group, d)
            z = torch.einsum("hgd,thd->hgt", qr, k[lo:hi]) * scale
            if softcap:
                z = softcap * torch.tanh(z / softcap)
            if slopes is not None:
                far = (torch.arange(lo, hi) - pos).abs().double()
                z = z - slopes.double().view(hkv, group, 1) * far
            p = torch.softmax(z, -1)
            out[row] = torch.einsum("hgt,thd->hgd", p, v[lo:hi]).reshape(hq, d)
            size[row] = torch.einsum("hgt,thd->hgd", p, v[lo:hi].abs()).reshape(hq, d)
    return out, size
