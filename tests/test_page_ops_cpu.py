"""The ragged page operators without a GPU: their float64 reference pinned, and every
refusal of the C ABI and of the binding before anything touches the device."""
import ctypes
import math
import types

import pytest
import torch

import oracle
import paged_gqa_decode_04_gb300 as pgd
from oracle import page_ops as ref
from page_ops_cases import Batch
from paged_gqa_decode_04_gb300 import _lib


def np_bits(t):
    return t.view(torch.uint16).numpy() if t.dtype == torch.bfloat16 else t.numpy()


@pytest.mark.parametrize("window", [0, 20])
def test_reference_attend_is_the_oracle_where_both_apply(window):
    b = Batch([40, 129, 64], [5, 5, 5], hkv=2, device="cpu")
    q = b.rows(8, packed=False)
    out, _ = ref.attend(q, b.k, b.v, None, None, b.cu, b.table, b.lens, 0.09, True, window)
    want, rc = oracle.decode_ex_f64(np_bits(q).reshape(3, 5, 8, 128), np_bits(b.k), np_bits(b.v),
                                    b.table.numpy(), b.len_t.numpy(), 0.09, window)
    assert rc == 0
    got = torch.stack([out[r] for r in range(15)]).numpy().reshape(want.shape)
    assert abs(got - want).max() < 1e-12


def test_reference_attend_closed_forms():
    b = Batch([30, 12], [4, 20], hkv=2, device="cpu")
    q = b.rows(4, packed=False)
    out, size = ref.attend(q, b.k, b.v, None, None, b.cu, b.table, b.lens, 0.0, False, 0)
    for s, rows in ((0, range(4)), (1, range(4, 24))):
        v = torch.stack([ref.values(b.v, None, *ref.place(b.table, 16, s, t))
                         for t in range(b.lens[s])])
        for r in rows:
            for h in range(4):
                assert torch.allclose(out[r][h], v[:, h // 2].mean(0), atol=1e-13, rtol=0)
                assert torch.allclose(size[r][h], v[:, h // 2].abs().mean(0), atol=1e-13, rtol=0)
    out, _ = ref.attend(q, b.k, b.v, None, None, b.cu, b.table, b.lens, 0.3, True, 0)
    for r in range(4, 12):                     # 20 queries over 12 tokens: 8 before the first
        assert torch.all(out[r] == 0)
    first = ref.values(b.v, None, *ref.place(b.table, 16, 1, 0))
    for h in range(4):
        assert torch.allclose(out[12][h], first[h // 2], atol=1e-13, rtol=0)


@pytest.mark.parametrize("interleaved", [False, True])
def test_reference_rotation(interleaved):
    """Position 0 is left alone, lengths are kept, and scores depend on the distance only."""
    g = torch.Generator().manual_seed(0)
    q, k = torch.randn((2, 3, 64), generator=g).double()
    rope = pgd.rope_table(50, 32)
    turn = lambda x, p: ref.norm_rotate(x, None, 0.0, rope, interleaved, p)[0]
    assert torch.equal(turn(q, 0), q)
    assert torch.equal(turn(q, 7)[:, 32:], q[:, 32:])
    assert torch.allclose(turn(q, 31).norm(dim=1), q.norm(dim=1), rtol=1e-6)
    a = (turn(q, 20) * turn(k, 13)).sum(1)
    c = (turn(q, 49) * turn(k, 42)).sum(1)
    assert torch.allclose(a, c, atol=1e-5)
    one = torch.zeros(1, 64).double()
    one[0, 0] = 1
    y = turn(one, 3)[0]
    assert math.isclose(float(y[0]), math.cos(3), abs_tol=1e-7)
    assert math.isclose(float(y[1 if interleaved else 16]), math.sin(3), abs_tol=1e-7)


def test_reference_norm():
    x = torch.tensor([[3.0, 4.0] * 8])
    w = torch.arange(16.0)
    y, _ = ref.norm_rotate(x, w, 0.0, None, False, 0)
    assert torch.allclose(y[0], x[0].double() / math.sqrt(12.5) * w.double())


def test_reference_codes():
    x = torch.tensor([0.0, 1.0, 1.9, 2.0, 440.0, 2.0 ** -6, 2.0 ** -9]).double()
    want = [2.0 ** -10, 2.0 ** -4, 2.0 ** -4, 2.0 ** -3, 16.0, 2.0 ** -10, 2.0 ** -10]
    assert ref.half_step(x, torch.float8_e4m3fn).tolist() == want
    codes = x.float().to(torch.float8_e4m3fn).double()
    assert torch.all((codes - x).abs() <= ref.half_step(x, torch.float8_e4m3fn))
    assert ref.half_step(x, torch.int8).tolist() == [0.5] * 7


def test_reference_block_scales():
    b = Batch([20, 16], [8, 16], hkv=1, pages="int8", scales="block", device="cpu")
    rows = torch.full((24, 1, 128), 1.27)
    rows[3] = 2.54                              # position 15, the first block's last slot
    rows[5, 0, 0] = float("inf")
    b.k_scale[b.table[0, 0]] = 0.005
    s = ref.block_scales(b.k, b.k_scale, rows, b.cu, b.table, b.lens)
    near = lambda x, y: abs(float(x) - y) < 1e-8
    assert near(s[int(b.table[0, 0])], 0.02) and near(s[int(b.table[0, 1])], 0.01)
    assert near(s[int(b.table[1, 0])], 0.01) and len(s) == 3
    b.k_scale[b.table[0, 0]] = 0.03
    s = ref.block_scales(b.k, b.k_scale, rows, b.cu, b.table, b.lens)
    assert near(s[int(b.table[0, 0])], 0.03)


def test_rope_table():
    t = pgd.rope_table(100000, 64, base=500000.0)
    assert t.shape == (100000, 2, 32) and t.dtype == torch.float32
    angle = 99999 * 500000.0 ** (-10 / 64)
    assert abs(float(t[99999, 0, 5]) - math.cos(angle)) < 2.0 ** -24 + 1e-9
    assert abs(float(t[99999, 1, 5]) - math.sin(angle)) < 2.0 ** -24 + 1e-9


# ------------------------------------------------------------------- refusals (C ABI)



def test_null_handles(lib):
    assert lib.paged_kv_write(None, 256, 256, 256, 256, 1, 256, 1, 256, 1, 256,
                              None) == _lib.PGD_ERR_ARG
    assert lib.paged_kv_read(None, 256, 256, 1, 256, 1, 256, 1, 256, None) == _lib.PGD_ERR_ARG
    assert lib.paged_qk_norm_rope_write(None, 256, 256, 256, 256, 2, 256, 256, 256, 256, 1, None,
                                        None, 1, 1e-6, None, 0, 0, 0, 256, 1, 256, 1, 256,
                                        None) == _lib.PGD_ERR_ARG
    assert lib.paged_gqa_attend(None, 256, 256, 1, 2, 256, 1, 256, 1, 256, 1, 0, 1.0, 256,
                                None) == _lib.PGD_ERR_ARG


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__

    __graft_entry__.build()
    return _lib.load()


def meta_pool(dtype=torch.bfloat16, hkv=2, d=128):
    return types.SimpleNamespace(q_dtype=dtype, head_dim=d, num_kv_heads=hkv,
                                 device=torch.device("cuda:0"))


def test_binding_refuses_tables():
    """Ranks, types and sizes of the tables, before the library is called."""
    from paged_gqa_decode_04_gb300 import kv_cache

    pool = meta_pool()
    cu = torch.zeros(3, dtype=torch.int32)
    table, lens = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    check = kv_cache._check_tables
    with pytest.raises(ValueError, match="cu_seqlens must be"):
        check(pool, cu[None], table, lens)
    with pytest.raises(ValueError, match="cu_seqlens must be"):
        check(pool, cu, table[0], lens)
    for bad in ((cu.long(), table, lens), (cu, table.long(), lens), (cu, table, lens.long())):
        with pytest.raises(TypeError, match="int32"):
            check(pool, *bad)
    with pytest.raises(ValueError, match="mismatch"):
        check(pool, cu[:2], table, lens)
    with pytest.raises(ValueError, match="mismatch"):
        check(pool, cu, table[:1], lens)
    with pytest.raises(ValueError, match="CUDA"):
        check(pool, cu, table, lens)


def test_binding_refuses_rows():
    from paged_gqa_decode_04_gb300 import kv_cache

    pool = meta_pool()
    x = torch.zeros(5, 2, 128, dtype=torch.bfloat16)
    check = kv_cache._check_rows
    for bad in (x[0], x[:, :1], x[..., :64]):
        with pytest.raises(ValueError, match="must be"):
            check(pool, "k", bad, 2)
    with pytest.raises(ValueError, match="must be"):
        check(pool, "v", x, 2, 4)
    with pytest.raises(TypeError, match="bfloat16"):
        check(pool, "k", x.float(), 2)
    with pytest.raises(ValueError, match="CUDA"):
        check(pool, "k", x, 2)
    with pytest.raises(ValueError, match="contiguous"):
        kv_cache._check_weight(pool, "q_weight", torch.ones(64))
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        kv_cache._check_weight(pool, "q_weight", torch.ones(128, dtype=torch.float16))
    with pytest.raises(ValueError, match="device"):
        kv_cache._check_weight(pool, "q_weight", torch.ones(128))
    assert kv_cache._check_weight(pool, "q_weight", None) is None
