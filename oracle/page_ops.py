"""Float64 reference of the ragged page operators (write, read, norm and rotation,
attention of many query tokens), straight from their definitions, on the CPU.

TEST INFRASTRUCTURE ONLY.  Tensors are torch CPU tensors; pools are given in their
stored type (float32, bfloat16, float8_e4m3fn or int8) and results are float64.
Sequence b owns rows cu[b] .. cu[b+1]-1, its last cached tokens.
"""
import torch

TOP = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}


def rows_of(cu, lens, b):
    """(packed row, position) of every new token of sequence b."""
    n = int(cu[b + 1]) - int(cu[b])
    return [(int(cu[b]) + i, int(lens[b]) - n + i) for i in range(n)]


def place(table, bs, b, pos):
    return int(table[b][pos // bs]), pos % bs


def half_step(x, dtype):
    """Half the spacing of the codes around x (float64 tensor, |x| <= top)."""
    if dtype == torch.int8:
        return torch.full_like(x, 0.5)
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    return torch.exp2(e - 4)


def values(pool, scale, blk, slot):
    """float64 [Hkv, D] of one slot."""
    x = pool[blk, slot].double()
    if scale is None:
        return x
    s = scale if scale.dim() == 1 else scale[blk]
    return x * s.double()[:, None]


def read(pool, scale, cu, table, lens):
    """{packed row: float64 [Hkv, D]}."""
    bs, out = pool.shape[1], {}
    for b in range(len(lens)):
        for row, pos in rows_of(cu, lens, b):
            out[row] = values(pool, scale, *place(table, bs, b, pos))
    return out


def block_scales(pool, scale, rows, cu, table, lens):
    """{block: float64 [Hkv]} of the blocks a write touches: the largest finite
    magnitude over the rows it stores there, and the scale before where the block holds
    earlier tokens of the sequence."""
    bs, top = pool.shape[1], TOP[pool.dtype]
    new = {}
    for b in range(len(lens)):
        for i, (row, pos) in enumerate(rows_of(cu, lens, b)):
            blk, slot = place(table, bs, b, pos)
            x = rows[row].double().abs()
            m = torch.where(torch.isfinite(x), x, 0.0).amax(-1) / top
            m = torch.where(m >= 2.0 ** -126, m, 0.0)
            if i == 0 and slot > 0:
                m = torch.maximum(m, scale[blk].double())
            new[blk] = torch.maximum(new[blk], m) if blk in new else m
    return new


def norm_rotate(x, weight, eps, rope, interleaved, pos):
    """float64 [heads, D] of one token; also sum of the magnitudes that met in each
    element (what a float32 evaluation's error is relative to)."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()
    size = x.abs()
    if rope is None:
        return x, size
    half = rope.shape[2]
    y, m = x.clone(), size.clone()
    for j in range(half):
        one, two = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        c, s = float(rope[pos, 0, j]), float(rope[pos, 1, j])
        y[:, one] = x[:, one] * c - x[:, two] * s
        y[:, two] = x[:, two] * c + x[:, one] * s
        m[:, one] = m[:, two] = size[:, one] + size[:, two]
    return y, m


def attend(q, k_pool, v_pool, k_scale, v_scale, cu, table, lens, scale, causal, window):
    """({row: out [Hq, D]}, {row: sum_t p_t |v_t| / sum_t p_t}), float64."""
    hq, hkv, bs = q.shape[1], k_pool.shape[2], k_pool.shape[1]
    group = hq // hkv
    out, size = {}, {}
    for b in range(len(lens)):
        L = int(lens[b])
        at = [place(table, bs, b, t) if int(table[b][t // bs]) >= 0 else None for t in range(L)]
        zero = torch.zeros(hkv, q.shape[2], dtype=torch.float64)
        k = torch.stack([values(k_pool, k_scale, *a) if a else zero for a in at]
                        ) if L else zero[None][:0]
        v = torch.stack([values(v_pool, v_scale, *a) if a else zero for a in at]
                        ) if L else zero[None][:0]
        for row, pos in rows_of(cu, lens, b):
            lo, hi = 0, L
            if causal:
                hi = pos + 1
                lo = max(0, pos - window + 1) if window else 0
            if hi <= lo:
                out[row] = torch.zeros(hq, q.shape[2], dtype=torch.float64)
                size[row] = out[row]
                continue
            qr = q[row].double().view(hkv, group, -1)
            z = torch.einsum("hgd,thd->hgt", qr, k[lo:hi]) * scale
            p = torch.softmax(z, -1)
            out[row] = torch.einsum("hgt,thd->hgd", p, v[lo:hi]).reshape(hq, -1)
            size[row] = torch.einsum("hgt,thd->hgd", p, v[lo:hi].abs()).reshape(hq, -1)
    return out, size
