"""What the decodes' binding refuses before the library is called, and the room that shared prefixes
need."""
import os
import subprocess
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


def test_results_of_prefixes_fit_what_the_largest_batch_is_given(tmp_path):
    """most_prefix_rows holds rows times prefix_splits of every batch up to its size, of any number
    of groups, and grows with the batch."""
    src = tmp_path / "m.cpp"
    src.write_text("""
#include <cstdio>
#include <initializer_list>
#include "attend_plan.h"
using namespace pgd::attend;
int main() {
    for (int sms : {148, 152})
        for (int hkv : {1, 2, 5, 8, 16})
            for (int per : {1, 3, 4, 8, 20, 64}) {          // rows of a sequence and KV head
                long long before = 0;
                for (int B = 1; B < 700; B += B < 80 ? 1 : 13) {
                    const long long heads = (long long)B * per * hkv;
                    const long long most = most_prefix_rows(heads, sms);
                    if (most < before) return printf("falls %d %d %d\\n", hkv, per, B), 1;
                    before = most;
                    for (int g = 1; g <= B; ++g)
                        if (heads * prefix_splits((long long)B * per, g, hkv, sms) > most)
                            return printf("small %d %d %d %d\\n", hkv, per, B, g), 1;
                }
            }
    printf("fits\\n");
}
""")
    inc = os.path.join(os.path.dirname(os.path.abspath(pgd.__file__)), "csrc")
    exe = tmp_path / "m"
    subprocess.run(["g++", "-std=c++17", "-O1", "-I" + inc, str(src), "-o", str(exe)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True)
    assert res.returncode == 0 and res.stdout == "fits\n", res.stdout
