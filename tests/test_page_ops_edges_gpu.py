"""Edges of the ragged page operators on the GPU, against their float64 definitions."""
import numpy as np
import pytest
import torch

import paged_gqa_decode_04_gb300 as pgd
from oracle import page_ops as ref
from page_ops_cases import Batch

pytestmark = pytest.mark.gpu


def check_rows(b, got, q, scale, causal, window, skip=()):
    """The rows of `got` against the definition, but for those in `skip`."""
    want, size = ref.attend(q, b.k, b.v, b.k_scale, b.v_scale, b.cu, b.table, b.lens, scale,
                            causal, window)
    got = got.cpu().double()
    for row, y in want.items():
        if row not in skip:
            # weights rounded to 16 bits (half a step, 2^-8), scores with float32 errors (below
            # 2^-13 of a weight, in numerator and denominator), the output rounded
            tol = 2.0 ** -8 * y.abs() + (2.0 ** -8 + 2.0 ** -12) * size[row]
            err = (got[row] - y).abs()
            assert torch.all(err <= tol), (row, float((err - tol).max()))


def rescaled_twice(pages, rows):
    """One sequence whose key tiles go in pairs: V's scales rise 1, 8, 16, 128, 256, .. and scores
    by 2^8.5 at 16, 256, ..: there the gain falls 16 times, from V's scales at the upper end of
    their range to the lower, and the maximum grows with it.  The tiles before then count 2^-9.5
    of the next ones' weight and scale, 2^-5.5 if the accumulator missed the gain."""
    L = 128 * 14 - 50
    b = Batch([L], [rows], hkv=1, pages=pages, scales="block", seed=rows)
    u = torch.randn(128, generator=b.g)
    u = u / u.abs().max()
    q = ((u + 0.02 * torch.randn((rows, 4, 128), generator=b.g)) * 0.5).bfloat16()
    top = ref.TOP[b.k.dtype]
    codes = u * top
    b.k[:] = (codes.round() if pages == "int8" else codes).to(b.k.dtype)
    codes = (0.5 + 0.5 * torch.rand(b.v.shape, generator=b.g)) * top
    b.v[:] = (codes.round() if pages == "int8" else codes).to(b.v.dtype)
    step = 8.5 * np.log(2) / float((q.double().mean((0, 1)) * b.k[0, 0, 0].double()).sum())
    pair = torch.arange(-(-L // 16)) // 16
    blk = b.table[0].long()[:len(pair)]
    b.k_scale[blk] = (step * (1 + pair // 2)).float()[:, None]
    b.v_scale[blk] = (15.9 * 2.0 ** -23 * 16.0 ** (pair // 2) * torch.where(pair % 2 == 1, 8.0, 1.0)
                      ).float()[:, None]
    return b, q


@pytest.mark.parametrize("pages", ["e4m3", "int8"])
@pytest.mark.parametrize("rows", [2, 70])
def test_attend_gain_and_maximum_change_in_one_tile(pages, rows):
    """700 sequences of the same pages and queries, so that no cluster shares the tiles."""
    b, q = rescaled_twice(pages, rows)
    n = 700
    cu = (torch.arange(n + 1) * rows).int().cuda()
    table, lens = b.table.repeat(n, 1).cuda(), b.len_t.repeat(n).cuda()
    pool = b.pool()
    for causal in (True, False):
        got = pgd.paged_gqa_attend(pool, q.repeat(n, 1, 1).cuda(), cu, table, lens, 1.0,
                                   causal=causal)
        assert pgd.paged_gqa_get_error(pool) == 0
        check_rows(b, got, q, 1.0, causal, 0)
        got = got.view(n, rows, 4, 128)
        assert torch.equal(got, got[:1].expand_as(got))
    pool.close()
