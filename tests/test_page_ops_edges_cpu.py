"""Refusals of the ragged page operators' binding that need no GPU."""
import types

import pytest
import torch

from paged_gqa_decode_04_gb300 import kv_cache


@pytest.mark.parametrize("B,columns", [(1, 2 ** 31), (1, 2 ** 32 + 4), (2 ** 32 + 1, 1)])
def test_binding_refuses_tables_beyond_an_int(B, columns):
    """Sizes that would wrap in the library's int arguments."""
    pool = types.SimpleNamespace(device=torch.device("cuda:0"))
    i32 = dict(dtype=torch.int32, device="meta")
    with pytest.raises(ValueError, match="2.31"):
        kv_cache._check_tables(pool, torch.empty(B + 1, **i32), torch.empty(B, columns, **i32),
                               torch.empty(B, **i32))
