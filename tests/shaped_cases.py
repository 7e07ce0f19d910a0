"""Batches whose sequences share prefixes in groups, and the bound that attention with shaped
scores is held to."""
import torch

from oracle import shaped as ref
from page_ops_cases import Batch


def alibi(heads, steep=8.0):
    return torch.exp2(-steep * torch.arange(1, heads + 1, dtype=torch.float64) / heads).float()


def tail(b, decode):
    """What f16 steps below its normal numbers add to an element for every token seen, over 8-bit
    pages.  A decode's weights, relative to the largest, are off by half a step of 2^-24, with
    block scales after V's scale is multiplied in: 2^-25 of the largest value, or of the largest
    code.  The attention's steps are 2^-28 of the largest weight times V's scale, or finer."""
    if b.v_scale is None:
        return 0.0
    top = {"e4m3": 448.0, "int8": 128.0}[b.pages]
    most = top * float(torch.nan_to_num(b.v_scale).max())
    if not decode:
        return 2.0 ** -29 * most
    return 2.0 ** -25 * (max(top, most) if b.v_scale.dim() == 2 else most)


def check_rows(b, got, q, scale, decode=False, **kw):
    """Rows of a bfloat16 result against the definition.  The output's rounding, and the
    weights', each half a bfloat16 step: 2^-8.  2^-12 for the rest: float32 sums, the cap's
    6.7e-7 of scores up to 220 in units of log 2 (below a cap of 200, whose tanh is 0.77 there;
    2^-21 beyond), a bias' rounding of 2^-24 of up to 2^10, the exponential's 2^-22, and parts
    joined in float32.  And the tail of weights in f16."""
    want, size = ref.attend(q, b.k, b.v, b.k_scale, b.v_scale, b.cu, b.table, b.lens, scale, **kw)
    low = tail(b, decode) * max(b.lens)
    for row, y in want.items():
        tol = 2.0 ** -8 * y.abs() + (2.0 ** -8 + 2.0 ** -12) * size[row] + low
        err = (got[row].double() - y).abs()
        assert torch.all(err <= tol), (row, float((err - tol).max()))
    return want


def share(b, groups, prefixes):
    """Make the sequences of `groups` ((first, end), ..) of a batch share their first tokens:
    whole blocks of the group's first sequence, the rest of the prefix copied.  The blocks that
    they held before are poisoned."""
    for (first, end), n in zip(groups, prefixes):
        members = [s for s in range(first, end) if b.lens[s]]
        for s in members[1:]:
            for i in range(n // b.bs):
                old = int(b.table[s][i])
                b.table[s][i] = b.table[members[0]][i]
                for p in (b.k, b.v):
                    bits = p.view(torch.uint8) if p.element_size() == 1 else p
                    bits[old] = {"e4m3": 0x7f, "int8": 0x80}.get(b.pages, float("nan"))
                if b.k_scale is not None and b.k_scale.dim() == 2:
                    b.k_scale[old] = b.v_scale[old] = float("nan")
            if n % b.bs:
                src, dst = int(b.table[members[0]][n // b.bs]), int(b.table[s][n // b.bs])
                for p in (b.k, b.v):
                    bits = p.view(torch.uint8) if p.element_size() == 1 else p
                    bits[dst, :n % b.bs] = bits[src, :n % b.bs]
                if b.k_scale is not None and b.k_scale.dim() == 2:
                    b.k_scale[dst], b.v_scale[dst] = b.k_scale[src], b.v_scale[src]


def shared_batch(own, groups, prefixes, q_len=1, **kw):
    """A batch of sequences with own[s] tokens behind their group's prefix (0: no tokens at
    all, not even the prefix), and the tables of the groups."""
    lens = list(own)
    for (first, end), n in zip(groups, prefixes):
        for s in range(first, end):
            lens[s] = own[s] + n if own[s] >= 0 else 0
    lens = [max(x, 0) for x in lens]
    b = Batch(lens, [q_len] * len(lens), **kw)
    share(b, groups, prefixes)
    return b


def group_tables(groups, prefixes, device="cuda"):
    cu = [g[0] for g in groups] + [groups[-1][1]]
    return (torch.tensor(cu, dtype=torch.int32, device=device),
            torch.tensor(list(prefixes), dtype=torch.int32, device=device))
