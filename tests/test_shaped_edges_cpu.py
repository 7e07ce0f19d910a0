"""What the decodes' binding refuses before the library is called."""
import types

import pytest
import torch

import paged_gqa_decode_04_gb300 as pgd
from test_page_ops_cpu import meta_pool


def test_decodes_refuse_outputs_and_workspaces():
    """Their type and size, and that they are where the pool is."""
    pool = meta_pool()
    q = torch.zeros(2, 1, 4, 128, dtype=torch.bfloat16)
    ws = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(TypeError, match="bfloat16"):
        pgd._check_out(pool, q, q.float(), ws)
    with pytest.raises(ValueError, match="smaller"):
        pgd._check_out(pool, q, q[:1], ws)
    with pytest.raises(ValueError, match="device"):
        pgd._check_out(pool, q, torch.empty_like(q), ws)
    on_cpu = types.SimpleNamespace(device=types.SimpleNamespace(index=-1))
    pgd._check_out(on_cpu, q, torch.empty(3, 4, 128, dtype=torch.bfloat16), ws)
    for bad in ((q, torch.zeros(512, dtype=torch.uint8)[::2]),
                (torch.empty(2, 1, 8, 128, dtype=torch.bfloat16)[:, :, ::2], ws)):
        with pytest.raises(ValueError, match="contiguous"):
            pgd._check_out(on_cpu, q, *bad)


def test_decodes_refuse_tables_elsewhere():
    pool = meta_pool()
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError, match="pool's device"):
        pgd._check_decode_args(pool, q, torch.zeros(2, 3, **i32), torch.zeros(2, **i32), 3)
