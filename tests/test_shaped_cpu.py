"""Attention with shaped scores and shared prefixes without a GPU: the float64 reference
pinned, the launch arithmetic, and what the binding refuses before the library is called."""
import ctypes
import math
import os
import shutil
import subprocess

import pytest
import torch

import paged_gqa_decode_04_gb300 as pgd
from oracle import page_ops, shaped
from page_ops_cases import Batch
from paged_gqa_decode_04_gb300 import _lib, kv_cache
from shaped_cases import alibi
from test_page_ops_cpu import meta_pool


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__

    __graft_entry__.build()
    return _lib.load()


def pin_batch():
    b = Batch([30, 12], [4, 12], hkv=2, device="cpu")
    return b, b.rows(4, packed=False)


def pools(b):
    return b.k, b.v, None, None, b.cu, b.table, b.lens


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 5), (False, 0)])
def test_reference_is_the_plain_one_where_nothing_is_shaped(causal, window):
    b, q = pin_batch()
    want, size = page_ops.attend(q, *pools(b), 0.2, causal, window)
    for kw in ({}, {"softcap": 1e9}, {"slopes": torch.zeros(4)},
               {"visible": torch.tensor([[-3, 1 << 30]] * 16)}):
        out, m = shaped.attend(q, *pools(b), 0.2, causal, window, **kw)
        for r, y in want.items():
            assert torch.allclose(out[r], y, atol=1e-12, rtol=0)
            assert torch.allclose(m[r], size[r], atol=1e-12, rtol=0)


def test_reference_by_hand():
    """Two tokens seen, in Python floats: cap, then bias, |p - t| on both sides of p."""
    b, q = pin_batch()
    sl = alibi(4)
    vis = torch.zeros(16, 2, dtype=torch.int32)
    vis[6] = torch.tensor([1, 3])                   # sequence 1, position 2: behind and itself
    vis[4] = torch.tensor([2, 4])                   # position 0: tokens ahead
    out, _ = shaped.attend(q, *pools(b), 0.7, causal=False, softcap=1.5, slopes=sl, visible=vis)
    for row, pos, seen in ((6, 2, (1, 2)), (4, 0, (2, 3))):
        for h in range(4):
            k, v = [[page_ops.values(p, None, *page_ops.place(b.table, 16, 1, t))[h // 2]
                     for t in seen] for p in (b.k, b.v)]
            s = [shaped.score(0.7 * float(q[row, h].double() @ x), 1.5, float(sl[h]), pos - t)
                 for x, t in zip(k, seen)]
            w = 1 / (1 + math.exp(s[1] - s[0]))
            assert torch.allclose(out[row][h], w * v[0] + (1 - w) * v[1], atol=1e-12, rtol=0)
    assert torch.all(out[5] == 0) and torch.all(out[0] == 0)


def test_reference_cap_bounds_scores():
    """Scores far above a cap of 2 are +-2 to within 4 e^-|s|: weights differ by e^4.  For
    |s| > 20 that is 9e-9, twice that for a weight's share, times |v| below 5: 1e-7."""
    b, q = pin_batch()
    out, _ = shaped.attend(q.float() * 100, *pools(b), 1.0, causal=False, softcap=2.0)
    k, v = [torch.stack([page_ops.values(p, None, *page_ops.place(b.table, 16, 0, t))[0]
                         for t in range(30)]) for p in (b.k, b.v)]
    z = k @ (q[0, 0].double() * 100)
    assert z.abs().min() > 20 and v.abs().max() < 5
    w = torch.softmax(2 * torch.sign(z), -1)
    assert torch.allclose(out[0][0], w @ v, atol=1e-7, rtol=0)


def test_parts_of_a_prefix(tmp_path):
    """Two key tiles a part or more, never more parts than splits; as many CTAs as fit."""
    src = tmp_path / "p.cpp"
    src.write_text("""
#include <cstdio>
#include <initializer_list>
#include "attend_plan.h"
using namespace pgd::attend;
int main() {
    for (int splits : {1, 3, 19, 64})
        for (int n : {0, 8, 128, 256, 257, 1024, 16384, 2147482000})
            printf("%d ", prefix_parts(n, splits));
    printf("%d %d %d %d %d\\n", prefix_splits(256, 1, 8, 152), prefix_splits(8, 4, 8, 152),
           prefix_splits(960, 1, 1, 152), prefix_splits(1 << 20, 1, 8, 152),
           prefix_splits(4, 1, 1, 152));
}
""")
    cxx = shutil.which("g++")
    inc = os.path.join(os.path.dirname(_lib.HERE), "paged_gqa_decode_04_gb300", "csrc")
    exe = tmp_path / "p"
    subprocess.run([cxx, "-std=c++17", "-I" + inc, str(src), "-o", str(exe)], check=True)
    got = list(map(int, subprocess.run([str(exe)], capture_output=True, text=True,
                                       check=True).stdout.split()))
    want = []
    for splits in (1, 3, 19, 64):
        for n in (0, 8, 128, 256, 257, 1024, 16384, 2147482000):
            want.append(min(splits, -(-n // 256)))
    assert got == want + [19, 4, 38, 1, 64]


def test_null_handles(lib):
    assert lib.paged_gqa_attend_shaped(None, 256, 256, 1, 2, 256, 1, 256, 1, 256, 1, 0, 1.0, 1.0,
                                       None, None, 256, None) == _lib.PGD_ERR_ARG
    assert lib.paged_gqa_decode_shaped(None, 256, 1, 1, 2, 256, 1, 256, 0, 1.0, 1.0, None, 256,
                                       256, 1 << 20, 0, None) == _lib.PGD_ERR_ARG
    assert lib.paged_gqa_decode_shared(None, 256, 1, 1, 2, 256, 256, 1, 256, 1, 256, 1.0, 0.0,
                                       None, 256, 256, 1 << 20, None) == _lib.PGD_ERR_ARG
    n = ctypes.c_size_t()
    assert lib.paged_gqa_workspace_size_shared(None, 1, 1, 2, 1, ctypes.byref(n)) \
        == _lib.PGD_ERR_ARG


def test_binding_refuses_slopes():
    pool = meta_pool()
    with pytest.raises(ValueError, match="contiguous"):
        kv_cache._slopes_ptr(pool, torch.ones(3), 4)
    with pytest.raises(ValueError, match="contiguous"):
        kv_cache._slopes_ptr(pool, torch.ones(8)[::2], 4)
    with pytest.raises(TypeError, match="float32"):
        kv_cache._slopes_ptr(pool, torch.ones(4, dtype=torch.bfloat16), 4)
    with pytest.raises(ValueError, match="device"):
        kv_cache._slopes_ptr(pool, torch.ones(4), 4)
    assert kv_cache._slopes_ptr(pool, None, 4) is None


def test_binding_refuses_shared_tables():
    pool = meta_pool()
    q = torch.zeros(4, 4, 128, dtype=torch.bfloat16)
    i32 = dict(dtype=torch.int32)
    cu, shared = torch.zeros(3, **i32), torch.zeros(2, **i32)
    table, lens = torch.zeros(4, 2, **i32), torch.zeros(4, **i32)
    call = pgd.paged_gqa_decode_shared
    with pytest.raises(ValueError, match="q must be"):
        call(pool, q[0], cu, shared, table, lens, 1.0)
    with pytest.raises(TypeError, match="bfloat16"):
        call(pool, q.float(), cu, shared, table, lens, 1.0)
    for bad in ((cu.long(), shared, table, lens), (cu, shared[None], table, lens),
                (cu, shared, table[:, ::2], lens), (cu, shared, table, lens.float())):
        with pytest.raises(ValueError, match="int32"):
            call(pool, q, *bad, 1.0)
    for bad in ((cu[:2], shared, table, lens), (cu, shared, table[:3], lens),
                (cu, shared, table, lens[:3])):
        with pytest.raises(ValueError, match="mismatch"):
            call(pool, q, *bad, 1.0)
    with pytest.raises(ValueError, match="device"):
        call(pool, q, cu, shared, table, lens, 1.0, out=torch.empty_like(q))
