"""Edges of the ragged page operators on the GPU, against their float64 definitions."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import paged_gqa_decode_04_gb300 as pgd
from oracle import page_ops as ref
from page_ops_cases import Batch, check_stored
from paged_gqa_decode_04_gb300 import _lib

pytestmark = pytest.mark.gpu

FORMS = [("bf16", "head", 64), ("bf16", "head", 128), ("e4m3", "head", 128),
         ("int8", "head", 128), ("e4m3", "block", 128), ("int8", "block", 128)]


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


# lengths, new rows, KV heads, columns of the table (0: as many as needed), logical block
# that is bad in the last sequence: pieces of both blocks of rows, one block, and pieces
# that clusters share
BAD_PAGES = [([40, 300], [40, 300], 2, 0, 9), ([40, 300], [40, 300], 2, 0, 18),
             ([129, 700], [20, 260], 2, 0, 33), ([9, 150], [9, 30], 2, 0, 8),
             ([2498], [4], 1, 0, 156), ([800, 700], [3, 150], 1, 4096, 38)]


@pytest.mark.parametrize("case", range(len(BAD_PAGES)))
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_attend_bad_page_reaches_only_the_rows_that_read_it(form, case):
    pages, scales, d = FORMS[form]
    lens, new, hkv, columns, at = BAD_PAGES[case]
    b = Batch(lens, new, hkv=hkv, d=d, pages=pages, scales=scales, seed=at)
    if columns:
        wide = torch.full((len(lens), columns - b.table.shape[1]), -1, dtype=torch.int32)
        b.table = torch.cat([b.table, wide], 1).contiguous()
    q = b.rows(4 * hkv)
    pool = b.pool()
    cu, table, len_t = b.where()
    s = len(lens) - 1
    table[s, at] = (-1, -2 ** 31, 2 ** 31 - 1, b.k.shape[0])[(form + case) % 4]
    for causal, window in ((True, 0), (True, 37), (False, 0)):
        got = pgd.paged_gqa_attend(pool, b.to(q), cu, table, len_t, 0.1, causal=causal,
                                   window=window)
        lost = set()
        for row, pos in ref.rows_of(b.cu, b.lens, s):
            lo, hi = (max(0, pos - window + 1) if window else 0, pos + 1) if causal \
                else (0, lens[s])
            if lo < min(16 * at + 16, lens[s]) and hi > 16 * at:
                lost.add(row)
        assert pgd.paged_gqa_get_error(pool) == (_lib.PGD_ERR_BLOCK_ID if lost else 0)
        nan = got.isnan().cpu()
        assert set(nan.any(2).any(1).nonzero()[:, 0].tolist()) == lost
        assert nan[sorted(lost)].all()
        check_rows(b, got, q, 0.1, causal, window, skip=lost)
    pool.close()


@pytest.mark.parametrize("pages", ["bf16", "e4m3"])
def test_attend_several_bad_pages(pages):
    """Windowed rows between two bad pages read neither of them."""
    b = Batch([900], [900], hkv=1, pages=pages, seed=3)
    q = b.rows(3)
    pool = b.pool()
    cu, table, len_t = b.where()
    for at in (2, 3, 30, 50):
        table[0, at] = -1
    got = pgd.paged_gqa_attend(pool, b.to(q), cu, table, len_t, 0.1, window=100)
    lost = {p for p in range(900) if any(16 * at <= p < 16 * at + 16 + 99 for at in (2, 3, 30, 50))}
    assert pgd.paged_gqa_get_error(pool) == _lib.PGD_ERR_BLOCK_ID
    nan = got.isnan().all(2).all(1).cpu()
    assert set(nan.nonzero()[:, 0].tolist()) == lost
    check_rows(b, got, q, 0.1, True, 100, skip=lost)
    pool.close()


@pytest.mark.parametrize("exponent", [23.6, 25.5])
@pytest.mark.parametrize("pages", ["e4m3", "int8"])
@pytest.mark.parametrize("rows", [2, 90])
def test_attend_tail_far_below_the_largest_weight(pages, rows, exponent):
    """One token with all but a 2^-exponent-th of every other token's weight, its value zero:
    the output is the tail's, c N w / (1 + N w).  Weights are held times 2^7 in 11 bits, in
    steps of 2^-24 at least: to half a step, max(2^-11 w, 2^-32)."""
    n = 3001
    b = Batch([n], [rows], hkv=1, pages=pages, seed=1)
    b.k.view(torch.uint8).zero_()
    first = int(b.table[0, 0])
    b.k[first, 0] = torch.ones(1, 128).to(b.k.dtype)
    c = 56.0 if pages == "e4m3" else 77.0
    b.v[:] = torch.full(b.v.shape, c).to(b.v.dtype)
    b.v[first, 0] = torch.zeros(1, 128).to(b.v.dtype)
    b.k_scale.fill_(1.0), b.v_scale.fill_(1.0)
    q = torch.full((rows, 4, 128), 1.0).bfloat16()
    scale = float(np.float32(exponent * np.log(2) / 128))
    pool = b.pool()
    got = pgd.paged_gqa_attend(pool, q.cuda(), *b.where(), scale, causal=False).cpu().double()
    assert pgd.paged_gqa_get_error(pool) == 0
    pool.close()
    w = 2.0 ** -exponent
    want = c * (n - 1) * w / (1 + (n - 1) * w)
    # the weights' rounding; float32 scores, exponentials and sums; the output's rounding
    tol = want * (max(2.0 ** -11, 2.0 ** -32 / w) + 2.0 ** -12 + 2.0 ** -8)
    assert (got - want).abs().max() <= tol


@pytest.mark.parametrize("pages,scales", [("bf16", "head"), ("e4m3", "block"), ("int8", "head")])
@pytest.mark.parametrize("new", [(150, 20, 200), (3, 2, 1)])
def test_attend_windows_shared_by_clusters(new, pages, scales):
    """Windows of a dozen key tiles behind a wide table, which clusters of 8 CTAs share."""
    b = Batch([2500, 2200, 1900], new, hkv=1, pages=pages, scales=scales, seed=new[0])
    wide = torch.full((3, 4096 - b.table.shape[1]), -1, dtype=torch.int32)
    b.table = torch.cat([b.table, wide], 1).contiguous()
    q = b.rows(4)
    pool = b.pool()
    for window in (1500, 200, 1):
        got = pgd.paged_gqa_attend(pool, b.to(q), *b.where(), 0.09, window=window)
        assert pgd.paged_gqa_get_error(pool) == 0
        check_rows(b, got, q, 0.09, True, window)
    pool.close()


@pytest.mark.parametrize("window", [2 ** 31, 2 ** 32 + 5, 2 ** 70])
def test_attend_windows_beyond_an_int(window):
    """A window that no length reaches is none, whatever its width; one below zero is refused."""
    b = Batch([200], [60], hkv=1, seed=2)
    q = b.rows(2)
    pool = b.pool()
    got = pgd.paged_gqa_attend(pool, b.to(q), *b.where(), 0.1, window=window)
    assert torch.equal(got, pgd.paged_gqa_attend(pool, b.to(q), *b.where(), 0.1))
    with pytest.raises(pgd.PagedGQAError, match="PGD_ERR_ARG"):
        pgd.paged_gqa_attend(pool, b.to(q), *b.where(), 0.1, window=-window)
    pool.close()


def test_idle_sequences_may_be_longer_than_the_rotation_table():
    """A sequence without new rows asks for no angle: nothing is reported for it, whatever its
    length is; one that is longer than its table's blocks still is."""
    b = Batch([20, 300, 30, 250], [20, 0, 30, 0], hkv=2, seed=7)
    q, k = b.rows(4), b.rows(2)
    rope = pgd.rope_table(30, 128)
    pool = b.pool()
    out = pgd.paged_qk_norm_rope_write(pool, b.to(q), b.to(k), b.to(k), *b.where(),
                                       rope=rope.cuda())
    assert pgd.paged_gqa_get_error(pool) == 0
    for s in (0, 2):
        for row, pos in ref.rows_of(b.cu, b.lens, s):
            y, m = ref.norm_rotate(q[row], None, 0.0, rope, False, pos)
            assert torch.all((out[row].cpu().double() - y).abs()
                             <= 2.0 ** -8 * y.abs() + 2.0 ** -20 * m)
    cu, table, lens = b.where()
    lens[1] = 16 * table.shape[1] + 1
    pgd.paged_qk_norm_rope_write(pool, b.to(q), b.to(k), b.to(k), cu, table, lens,
                                 rope=rope.cuda())
    assert pgd.paged_gqa_get_error(pool) == _lib.PGD_ERR_SEQ_LEN
    pool.close()


@pytest.mark.parametrize("pages", ["e4m3", "int8"])
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -149, 2.0 ** -130, 2.0 ** -127])
def test_write_scales_too_small_to_divide_by(pages, scale):
    """A scale below the smallest normal number counts as zero: codes 0, for zeros too."""
    b = Batch([20, 16], [20, 16], hkv=2, pages=pages)
    k = b.rows(2)
    k[3], k[5, 0, :7] = 0, 0
    b.k_scale[0], b.v_scale[1] = scale, scale
    pool = b.pool()
    pgd.paged_kv_write(pool, b.to(k), b.to(k), *b.where())
    assert pgd.paged_gqa_get_error(pool) == 0
    pool.close()
    for s in range(2):
        for _, pos in ref.rows_of(b.cu, b.lens, s):
            blk, slot = ref.place(b.table, 16, s, pos)
            assert torch.all(b.dk.cpu()[blk, slot, 0].float() == 0)
            assert torch.all(b.dv.cpu()[blk, slot, 1].float() == 0)
            assert b.dk.cpu()[blk, slot, 1].float().isfinite().all()


@pytest.mark.parametrize("pages", ["e4m3", "int8"])
def test_write_behind_tokens_of_a_scale_too_small(pages):
    """A block whose scale so far is below the smallest normal number: zero rows keep it and
    get codes 0, others set a new one."""
    b = Batch([20, 20], [8, 8], hkv=2, pages=pages, scales="block")
    k = b.rows(2)
    k[:8] = 0
    for s in range(2):
        b.k_scale[b.table[s, 0].long()] = 2.0 ** -140
    pool = b.pool()
    pgd.paged_kv_write(pool, b.to(k), b.to(k), *b.where())
    assert pgd.paged_gqa_get_error(pool) == 0
    pool.close()
    got = b.dk.cpu()
    for pos in range(12, 20):
        blk, slot = ref.place(b.table, 16, 0, pos)
        assert torch.all(got[blk, slot].float() == 0)
        blk, slot = ref.place(b.table, 16, 1, pos)
        s = b.dks.cpu()[blk].double()[:, None]
        x = k[8 + pos - 12].double()
        half = ref.half_step((x / s).clamp(-ref.TOP[got.dtype], ref.TOP[got.dtype]), got.dtype)
        assert torch.all((got[blk, slot].double() * s - x).abs()
                         <= s * half * (1 + 2.0 ** -20) + 2.0 ** -22 * x.abs())


@pytest.mark.parametrize("scale", [2.5e38, -3.4e38])
def test_attend_refuses_scales_that_overflow(scale):
    """Scores are held in units of log 2: a scale that is infinite there is refused."""
    b = Batch([20], [4], hkv=1, seed=1)
    q = torch.zeros(4, 2, 128).bfloat16().cuda()
    pool = b.pool()
    with pytest.raises(pgd.PagedGQAError, match="PGD_ERR_ARG"):
        pgd.paged_gqa_attend(pool, q, *b.where(), scale)
    largest = pgd.paged_gqa_attend(pool, q, *b.where(), 2.3e38 * np.sign(scale))
    assert torch.equal(largest, pgd.paged_gqa_attend(pool, q, *b.where(), 0.0))
    pool.close()


def many(B, seed, **kw):
    """B sequences, most of them of a few tokens, with runs of sequences that have no new rows
    at both ends and in the middle."""
    r = np.random.default_rng(seed)
    lens = r.integers(0, 24, size=B)
    lens[r.integers(0, B, size=3)] = (150, 300, 90)
    new = np.minimum(lens, r.integers(0, 6, size=B))
    new[r.integers(0, B, size=2)] = 300
    new = np.minimum(new, lens)
    for lo, n in ((0, 3), (B // 2, B // 5), (B - 2, 2)):
        new[lo:lo + n] = 0
    return Batch(lens.tolist(), new.tolist(), bs=8, seed=seed, pad=3, **kw)


@pytest.mark.parametrize("B", [31, 33, 64, 1030])
@pytest.mark.parametrize("pages,scales", [("bf16", "head"), ("e4m3", "block")])
def test_batches_of_many_sequences(B, pages, scales):
    """Up to three rounds of the search for a row's sequence, through every operator."""
    b = many(B, B, hkv=1, pages=pages, scales=scales)
    rope = pgd.rope_table(300, 16)
    q, k, v = b.rows(2), b.rows(1), b.rows(1)
    rows = b.held_rows()
    pool = b.pool()
    out = pgd.paged_qk_norm_rope_write(pool, b.to(q), b.to(k), b.to(v), *b.where(),
                                       rope=rope.cuda()).cpu().double()
    assert pgd.paged_gqa_get_error(pool) == 0
    want, size = {}, {}
    for s in range(B):
        for row, pos in ref.rows_of(b.cu, b.lens, s):
            y, m = ref.norm_rotate(q[row], None, 0.0, rope, False, pos)
            assert torch.all((out[row] - y).abs() <= 2.0 ** -8 * y.abs() + 2.0 ** -20 * m)
            want[row], size[row] = ref.norm_rotate(k[row], None, 0.0, rope, False, pos)
    check_stored(b, "k", want, size, b.dk, b.dks, 2.0 ** -20)
    same = {r: v[r].double() for r in rows}
    check_stored(b, "v", same, {r: y.abs() for r, y in same.items()}, b.dv, b.dvs, 0.0)
    pool.close()
    pool = b.pool()                                   # the pages as they were
    pgd.paged_kv_write(pool, b.to(k), b.to(v), *b.where())
    assert pgd.paged_gqa_get_error(pool) == 0
    for name, x, after, sc in (("k", k, b.dk, b.dks), ("v", v, b.dv, b.dvs)):
        want = {r: x[r].double() for r in rows}
        check_stored(b, name, want, {r: y.abs() for r, y in want.items()}, after, sc, 0.0)
    pool.close()
    pool = b.pool()
    got = pgd.paged_kv_read(pool, b.total, *b.where())
    assert pgd.paged_gqa_get_error(pool) == 0
    for x, p, s in zip(got, (b.k, b.v), (b.k_scale, b.v_scale)):
        for r, y in ref.read(p, s, b.cu, b.table, b.lens).items():
            assert torch.all((x[r].cpu().double() - y).abs() <= (2.0 ** -8 + 2.0 ** -23) * y.abs())
    for causal in (True, False):
        o = pgd.paged_gqa_attend(pool, b.to(q), *b.where(), 0.09, causal=causal)
        assert pgd.paged_gqa_get_error(pool) == 0
        check_rows(b, o, q, 0.09, causal, 0)
    pool.close()


@pytest.mark.parametrize("lens,new,columns", [([1500, 700], [300, 700], 0), ([2600], [3], 0),
                                              ([900, 33], [150, 33], 8192)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1000)])
def test_attend_heads_of_64_over_many_tiles(lens, new, columns, causal, window):
    """The ring of eight tiles in several turns, with and without clusters."""
    b = Batch(lens, new, hkv=1, d=64, seed=len(lens) + columns)
    if columns:
        wide = torch.full((len(lens), columns - b.table.shape[1]), -1, dtype=torch.int32)
        b.table = torch.cat([b.table, wide], 1).contiguous()
    q = b.rows(4)
    pool = b.pool()
    got = pgd.paged_gqa_attend(pool, b.to(q), *b.where(), 0.125, causal=causal, window=window)
    assert pgd.paged_gqa_get_error(pool) == 0
    check_rows(b, got, q, 0.125, causal, window)
    pool.close()


CAPTURED_FIRST = """
import sys
sys.path[:0] = [%r, %r]
import torch
import paged_gqa_decode_04_gb300 as pgd
from page_ops_cases import Batch, bits
b = Batch([300, 40], [100, 40], hkv=2, pages=%r, scales="block", seed=1)
q, k = b.to(b.rows(8)), b.to(b.rows(2))
pool, where = b.pool(), b.where()
out = torch.zeros_like(q, memory_format=torch.contiguous_format)
qo = torch.zeros_like(out)
kv = [torch.zeros((b.total, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
rope = pgd.rope_table(300, 128, device="cuda")
def step(s):
    pgd.paged_qk_norm_rope_write(pool, q, k, k, *where, rope=rope, q_out=qo, stream=s)
    pgd.paged_gqa_attend(pool, qo, *where, 0.09, out=out, stream=s)
    pgd.paged_kv_read(pool, b.total, *where, out=kv, stream=s)
torch.cuda.synchronize()
g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
with torch.cuda.graph(g, stream=s):
    step(s)
g.replay()
torch.cuda.synchronize()
first = [t.clone() for t in (out, qo, *kv)]
pool = b.pool()                                       # the pages as they were, other buffers
step(s)
s.synchronize()
assert pgd.paged_gqa_get_error(pool) == 0
for x, y in zip(first, (out, qo, *kv)):
    assert x.abs().sum() > 0 and torch.equal(bits(x), bits(y))
print("same")
"""


@pytest.mark.parametrize("pages", ["bf16", "e4m3"])
def test_first_calls_of_a_process_are_captured(pages):
    """The library's first calls inside a graph capture, replayed: what eager calls give."""
    here = os.path.dirname(os.path.abspath(__file__))
    code = CAPTURED_FIRST % (os.path.dirname(here), here, pages)
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=240)
    assert res.returncode == 0 and res.stdout.strip() == "same", res.stderr[-2000:]


def test_waits_that_run_out_leave_the_attention_usable():
    """The attention's bounded waits give up, each by its own limit or because another thread
    did; the status is read and cleared, and the next call is right."""
    b = Batch([300, 40], [100, 40], hkv=2, seed=1)
    q = b.rows(8)
    pool = b.pool()
    s = torch.cuda.current_stream().cuda_stream
    for limit_us in (1, 1000):
        assert _lib.load().paged_gqa_selftest_wait_timeout(pool.handle, limit_us, s) == 0
        assert pgd.paged_gqa_get_error(pool) == _lib.PGD_ERR_TIMEOUT
        got = pgd.paged_gqa_attend(pool, b.to(q), *b.where(), 0.09)
        assert pgd.paged_gqa_get_error(pool) == 0
        check_rows(b, got, q, 0.09, True, 0)
    pool.close()


@pytest.mark.parametrize("pages", ["bf16", "e4m3"])
def test_prompts_and_steps_on_the_block_manager_s_tables(pages):
    """Prompts and steps of single tokens written and attended to through the tables of the block
    manager (a position reserved for each token), with a fork whose shared block is copied."""
    lens, bs, blocks = [37, 5, 64], 16, 24
    b = Batch(lens, lens, hkv=2, bs=bs, pages=pages, scales="block", seed=11)
    shape = (blocks, bs, 2, 128)
    b.k, b.v = torch.zeros(shape, dtype=b.k.dtype), torch.zeros(shape, dtype=b.v.dtype)
    if pages == "e4m3":
        b.k_scale, b.v_scale = torch.zeros(blocks, 2), torch.zeros(blocks, 2)
    pool = b.pool()
    kvm = pgd.KVBlockManager(blocks, bs, max_seqs=4, max_blocks_per_seq=8)
    for s, n in enumerate(lens):
        kvm.add_sequence(s)
        for _ in range(n):
            assert kvm.append_slots([s])[1] == []
    kvm.fork(0, 3)
    q, k, v = b.rows(8), b.rows(2), b.rows(2)
    rope = pgd.rope_table(128, 128, device="cuda")

    def step(q, k, v, cu, seqs, causal_rows):
        table, lens = [torch.from_numpy(x) for x in kvm.block_tables(seqs)]
        where = [cu.cuda(), table.cuda(), lens.cuda()]
        qo = pgd.paged_qk_norm_rope_write(pool, q.cuda(), k.cuda(), v.cuda(), *where, rope=rope)
        got = pgd.paged_gqa_attend(pool, qo, *where, 0.09)
        assert pgd.paged_gqa_get_error(pool) == 0
        now = [t.cpu() if t is not None else None for t in (b.dk, b.dv, b.dks, b.dvs)]
        want, size = ref.attend(qo.cpu(), *now, cu, table, lens, 0.09, True, 0)
        assert len(want) == causal_rows
        for row, y in want.items():
            tol = 2.0 ** -8 * y.abs() + (2.0 ** -8 + 2.0 ** -12) * size[row]
            assert torch.all((got[row].cpu().double() - y).abs() <= tol)
        return now, table, lens

    step(q, k, v, b.cu, [0, 1, 2], sum(lens))
    q, k, v = [torch.randn((4, h, 128), generator=b.g).bfloat16() for h in (8, 2, 2)]
    slots, copies = kvm.append_slots([0, 1, 2, 3])
    assert len(copies) == 1                              # the last block that 0 and 3 share
    src, dst = (torch.tensor(c, dtype=torch.int32, device="cuda") for c in zip(*copies))
    pgd.paged_kv_copy_blocks(pool, src, dst)
    now, table, lens = step(q, k, v, torch.arange(5).int(), [0, 1, 2, 3], 4)
    for s in range(4):                                   # the step's rows where the manager says
        blk, slot = ref.place(table, bs, s, int(lens[s]) - 1)
        assert blk * bs + slot == int(slots[s])
        stored = ref.values(now[1], now[3], blk, slot)
        # within half a step of the type, at the widest spacing of e4m3 (32 of 448)
        most = v[s].double().abs() if now[3] is None else 16 * now[3][blk].double()[:, None]
        assert torch.all((stored - v[s].double()).abs() <= most * (1 + 2.0 ** -20))
        if now[3] is None:
            assert torch.equal(stored, v[s].double())
    kvm.close()
    pool.close()
