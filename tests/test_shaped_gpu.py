"""Attention with shaped scores (soft cap, distance bias, visible ranges) and decode with shared
prefixes on the GPU, against their float64 definitions."""
import os
import subprocess
import sys

import pytest
import torch

import paged_gqa_decode_04_gb300 as pgd
from oracle import page_ops as ref
from oracle import shaped
from page_ops_cases import Batch
from paged_gqa_decode_04_gb300 import _lib
from shaped_cases import alibi, check_rows, group_tables, shared_batch

pytestmark = pytest.mark.gpu

LENS = [1, 40, 0, 129, 33, 64, 17, 300]
NEW = [1, 0, 0, 129, 20, 7, 1, 45]
FORMS = [("bf16", "head", 64), ("bf16", "head", 128), ("e4m3", "head", 128),
         ("int8", "head", 128), ("e4m3", "block", 128), ("int8", "block", 128)]
SHAPES = {"cap": dict(softcap=3.0), "bias": dict(slopes=True),
          "both": dict(softcap=30.0, slopes=True), "mask": {}}


def ok(pool):
    assert pgd.paged_gqa_get_error(pool) == 0


def shape_of(name, hq):
    kw = dict(SHAPES[name])
    if kw.get("slopes"):
        kw["slopes"] = alibi(hq)
    return kw


def documents(b, size, causal=True):
    """Ranges of documents of `size` tokens packed into each sequence."""
    vis = torch.zeros(b.total, 2, dtype=torch.int32)
    for s in range(len(b.lens)):
        for row, pos in ref.rows_of(b.cu, b.lens, s):
            vis[row, 0] = max(pos, 0) // size * size
            vis[row, 1] = vis[row, 0] + size
    return vis


def prefixes(b, part):
    """[0, max(p + 1, prefix)) with prefix = part of the length."""
    vis = torch.zeros(b.total, 2, dtype=torch.int32)
    for s in range(len(b.lens)):
        for row, pos in ref.rows_of(b.cu, b.lens, s):
            vis[row, 1] = max(pos + 1, int(b.lens[s] * part))
    return vis


def run_attend(b, q, scale, causal=True, window=0, softcap=0.0, slopes=None, visible=None,
               out=None):
    pool = b.pool()
    got = pgd.paged_gqa_attend(
        pool, b.to(q), *b.where(), scale, causal=causal, window=window, softcap=softcap,
        slopes=None if slopes is None else slopes.cuda(),
        visible=None if visible is None else visible.cuda(), out=out)
    ok(pool)
    pool.close()
    return got.cpu()


def check_attend(b, hq, scale=None, q=None, out=None, **kw):
    q = b.rows(hq) * 3 if q is None else q
    scale = b.d ** -0.5 if scale is None else scale
    got = run_attend(b, q, scale, out=out, **kw)
    check_rows(b, got, q, scale, **kw)
    return got


@pytest.mark.parametrize("bs", [8, 64, 256])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("pages,scales,d", FORMS)
def test_attend(pages, scales, d, shape, bs):
    """Causal, windowed, cross and masked, and rows behind the last sequence left alone."""
    for i, (causal, window, mask) in enumerate([(True, 0, None), (True, 30, None),
                                                (False, 0, None), (True, 0, "docs"),
                                                (False, 0, "docs"), (False, 0, "prefix")]):
        if shape == "mask" and not mask:
            continue
        b = Batch(LENS, NEW, hkv=2, d=d, bs=bs, pages=pages, scales=scales, seed=bs + i, pad=2)
        vis = {"docs": documents(b, 50), "prefix": prefixes(b, 0.5)}.get(mask)
        out = torch.full((b.total, 6, d), 7.0, dtype=b.act, device="cuda")
        got = check_attend(b, 6, causal=causal, window=window, visible=vis, out=out,
                           **shape_of(shape, 6))
        assert torch.all(got[int(b.cu[-1]):] == 7)


@pytest.mark.parametrize("shape", ["cap", "bias", "both", "mask"])
@pytest.mark.parametrize("pages,scales", [("bf16", "head"), ("e4m3", "block"), ("int8", "head")])
def test_attend_many_tiles(pages, scales, shape):
    """Several key tiles and row blocks a head: causal, cross, a window, documents longer and
    shorter than a tile, a prefix."""
    for causal, window, mask in ((True, 0, None), (False, 0, None), (True, 200, None),
                                 (True, 0, 300), (False, 0, 37), (False, 0, "prefix")):
        if shape == "mask" and not mask:
            continue
        b = Batch([1000, 517, 2], [500, 517, 1], hkv=1, bs=32, pages=pages, scales=scales,
                  seed=9)
        vis = None
        if mask:
            vis = prefixes(b, 0.7) if mask == "prefix" else documents(b, mask)
        check_attend(b, 3, causal=causal, window=window, visible=vis, **shape_of(shape, 3))


@pytest.mark.parametrize("hkv,group", [(1, 1), (5, 1), (1, 40), (2, 7), (3, 130)])
def test_attend_heads(hkv, group):
    for kw in (dict(softcap=5.0), dict(slopes=alibi(hkv * group)), {}):
        b = Batch([70, 9, 131], [5, 9, 90], hkv=hkv, seed=group)
        vis = documents(b, 40)
        check_attend(b, hkv * group, visible=vis, **kw)


@pytest.mark.parametrize("pages,scales", [("bf16", "head"), ("e4m3", "block")])
@pytest.mark.parametrize("B", [3, 12, 26])
def test_attend_clusters(B, pages, scales):
    """Wide tables make CTAs of a cluster share a piece of rows."""
    b = Batch([700 + 16 * i for i in range(B)], [(150, 20, 200, 90)[i % 4] for i in range(B)],
              hkv=1, pages=pages, scales=scales, seed=B)
    wide = torch.full((B, 4096 - b.table.shape[1]), -1, dtype=torch.int32)
    b.table = torch.cat([b.table, wide], 1).contiguous()
    check_attend(b, 4, softcap=4.0)
    check_attend(b, 4, causal=False, slopes=alibi(4))
    check_attend(b, 4, visible=documents(b, 333))


def test_attend_ranges_of_any_values():
    """Ranges that are empty, turned round, negative or far too long; rows that see nothing
    beside rows that see all; every row of a sequence hidden."""
    b = Batch([300, 40, 200], [300, 40, 200], hkv=2, seed=3)
    vis = torch.zeros(b.total, 2, dtype=torch.int32)
    g = torch.Generator().manual_seed(1)
    vis[:300] = torch.randint(-50, 400, (300, 2), generator=g)
    vis[:300:7, 1] = 2 ** 31 - 1
    vis[:300:11, 0] = -2 ** 31
    vis[300:340] = torch.tensor([5, 5])
    vis[340:] = torch.tensor([-2 ** 31, 2 ** 31 - 1])
    vis[345] = torch.tensor([200, 100])
    for causal in (True, False):
        for kw in ({}, dict(softcap=2.0), dict(slopes=alibi(4))):
            got = check_attend(b, 4, causal=causal, visible=vis, **kw)
            assert torch.all(got[300:340] == 0) and torch.all(got[345] == 0)


@pytest.mark.parametrize("pages", ["bf16", "e4m3"])
def test_attend_nothing_outside_the_ranges_is_read(pages):
    """Pages before and behind what any row sees may be gone, and hold NaN."""
    b = Batch([400, 333], [100, 333], hkv=2, pages=pages, seed=2)
    vis = torch.tensor([[150, 260]], dtype=torch.int32).repeat(b.total, 1)
    for s in range(2):
        for i in list(range(0, 150 // 16)) + list(range(-(-260 // 16), -(-b.lens[s] // 16))):
            blk = int(b.table[s][i])
            for p in (b.k, b.v):
                bits = p.view(torch.uint8) if p.element_size() == 1 else p
                bits[blk] = 0x7f if pages == "e4m3" else float("nan")
            b.table[s][i] = -1
        for t in list(range(144, 150)) + list(range(260, 272)):
            blk, slot = ref.place(b.table, 16, s, t)
            for p in (b.k, b.v):
                bits = p.view(torch.uint8) if p.element_size() == 1 else p
                bits[blk, slot] = 0x7f if pages == "e4m3" else float("nan")
    for kw in ({}, dict(softcap=2.0), dict(slopes=alibi(4))):
        check_attend(b, 4, causal=False, visible=vis, **kw)


def test_attend_sharp_scores():
    """Scores near +-900, capped where they bend and where they do not, scales of each sign."""
    b = Batch([600], [140], hkv=1, seed=4)
    q = (b.rows(4).float() * 9).to(torch.bfloat16)
    for cap in (1.0, 50.0, 1000.0, 2.0 ** 40):
        check_attend(b, 4, q=q, scale=2.0, softcap=cap, causal=False)
        check_attend(b, 4, q=q, scale=-1.0, softcap=cap)
    check_attend(b, 4, q=q, scale=0.0, softcap=10.0)
    check_attend(b, 4, q=q, scale=0.0, slopes=alibi(4))


def test_attend_steep_flat_and_negative_slopes():
    """Slopes from 0 to 8 a token, and below 0, where the farthest tokens weigh most.  The bias
    is rounded at its size: 300 tokens at slope 0.5 in units of log 2 is below 2^8, so 2^-16 of
    a weight, within the bound's 2^-12."""
    b = Batch([300, 280], [130, 280], hkv=2, seed=5)
    sl = torch.tensor([0.0, 8.0, 1.0, 2.0 ** -8, -0.5, -2.0 ** -6])
    check_attend(b, 6, slopes=sl)
    check_attend(b, 6, slopes=sl, causal=False)


def test_attend_masked_keys_may_hold_anything():
    """Infinities and NaN in keys that some rows do not see: only those that do suffer."""
    b = Batch([200], [200], hkv=1, seed=6)
    blk, slot = ref.place(b.table, 16, 0, 150)
    b.k[blk, slot] = float("nan")
    vis = torch.tensor([[0, 150]], dtype=torch.int32).repeat(200, 1)
    vis[60] = torch.tensor([140, 160])
    b2 = Batch([200], [200], hkv=1, seed=6)
    q = b2.rows(2)
    for kw in ({}, dict(softcap=4.0), dict(slopes=alibi(2))):
        got = run_attend(b, q, 0.1, causal=False, visible=vis, **kw)
        assert torch.all(got[60].isnan())
        want, size = shaped.attend(q, b2.k, b2.v, None, None, b2.cu, b2.table, b2.lens, 0.1,
                                   causal=False, visible=vis, **kw)
        for r in range(200):
            if r != 60:
                tol = 2.0 ** -8 * want[r].abs() + (2.0 ** -8 + 2.0 ** -12) * size[r]
                assert torch.all((got[r].double() - want[r]).abs() <= tol)


@pytest.mark.parametrize("pages,scales,d", FORMS)
@pytest.mark.parametrize("cap", [2.0, 55.0, 56.0, 200.0])
def test_attend_caps_and_where_scores_lie(cap, pages, scales, d):
    """Caps on both sides of the one from which on weights are relative to the row's maximum;
    scores far below the cap, about it and beyond it, in some rows and in all; rows whose scores
    are all at the lower end of the cap."""
    b = Batch([260, 140], [150, 140], hkv=1, d=d, pages=pages, scales=scales, seed=11)
    q = b.rows(3).float()
    size = torch.tensor([0.02, 1.0, 8.0, 60.0])[torch.arange(b.total) % 4]
    size[200:] = 0.1
    q = (q * size[:, None, None] * (2.0 if b.k_scale is None else 1.0)).to(torch.bfloat16)
    check_attend(b, 3, q=q, scale=0.3, softcap=cap)
    check_attend(b, 3, q=q, scale=0.3, softcap=cap, slopes=alibi(3), causal=False)
    # every key the same: all scores of a row are equal, most at -cap or cap
    b = Batch([130], [130], hkv=1, d=d, pages="bf16", seed=12)
    b.k[:] = torch.where(b.k.isnan(), b.k, torch.ones((), dtype=b.k.dtype))
    q = -torch.ones(130, 2, d, dtype=torch.bfloat16)
    q[::3] = 0.01
    check_attend(b, 2, q=q, scale=40.0, softcap=cap)


def test_attend_values_of_any_usual_size():
    """Values of 2^-20 and 2^30 keep their precision under a fixed reference."""
    for size in (2.0 ** -20, 2.0 ** 30):
        b = Batch([150], [150], hkv=1, seed=13)
        b.v *= size
        check_attend(b, 2, softcap=50.0)
        check_attend(b, 2, softcap=50.0, causal=False)


def test_attend_rows_of_a_wide_projection():
    """Query rows as views, their stride not a power of two, and out given."""
    b = Batch([90, 200], [90, 33], hkv=2, seed=14)
    wide = torch.randn(b.total, 6 + 5, 128, generator=b.g).to(torch.bfloat16)
    q = wide[:, 3:9]
    out = torch.full((b.total, 6, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    got = check_attend(b, 6, q=q, softcap=4.0, slopes=alibi(6), out=out)
    assert torch.equal(got, out.cpu())


CAPTURED_FIRST = """
import sys
sys.path[:0] = [%r, %r]
import torch
import paged_gqa_decode_04_gb300 as pgd
from shaped_cases import alibi, group_tables, shared_batch
groups, n = [(0, 3)], [300]
b = shared_batch([20, 7, 64], groups, n, hkv=2, pages=%r, scales="block", seed=7)
pool = b.pool()
q = b.rows(4, packed=False).cuda()
cu, table, lens = b.where()
cg, shared = group_tables(groups, n)
sl = alibi(4).cuda()
ws, wd = pgd.alloc_workspace_shared(pool, 3, 1, 4, 1), pgd.alloc_workspace(pool, 3, 4)
outs = [torch.zeros_like(q) for _ in range(4)]
def step(s):
    kw = dict(softcap=5.0, stream=s)
    pgd.paged_gqa_attend(pool, q, cu, table, lens, 0.1, out=outs[0], **kw)
    pgd.paged_gqa_attend(pool, q, cu, table, lens, 0.1, slopes=sl, out=outs[1], stream=s)
    pgd.paged_gqa_decode_ex(pool, q.view(3, 1, 4, 128), table, lens, 0.1, slopes=sl, workspace=wd,
                            out=outs[2].view(3, 1, 4, 128), **kw)
    pgd.paged_gqa_decode_shared(pool, q, cg, shared, table, lens, 0.1, workspace=ws,
                                out=outs[3], **kw)
torch.cuda.synchronize()
g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
with torch.cuda.graph(g, stream=s):
    step(s)
g.replay()
torch.cuda.synchronize()
first = [t.clone() for t in outs]
for t in outs: t.zero_()
torch.cuda.synchronize()
step(s)
s.synchronize()
assert pgd.paged_gqa_get_error(pool) == 0
for x, y in zip(first, outs):
    assert x.abs().sum() > 0 and torch.equal(x, y)
print("same")
"""


@pytest.mark.parametrize("pages", ["bf16", "e4m3"])
def test_first_calls_of_a_process_are_captured(pages):
    """The first calls of a process inside a graph capture, replayed: what eager calls give."""
    here = os.path.dirname(os.path.abspath(__file__))
    code = CAPTURED_FIRST % (os.path.dirname(here), here, pages)
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=240)
    assert res.returncode == 0 and res.stdout.strip() == "same", res.stderr[-2000:]


def test_many_groups_and_sequences():
    """More groups than a warp looks at, of one to five sequences, some without tokens."""
    g = torch.Generator().manual_seed(3)
    groups, n, own, at = [], [], [], 0
    for i in range(70):
        size = i % 5 + 1
        groups.append((at, at + size))
        n.append(int(torch.randint(0, 60, (1,), generator=g)))
        own += [(-1 if (at + k) % 13 == 5 else int(torch.randint(1, 30, (1,), generator=g)))
                for k in range(size)]
        at += size
    b = shared_batch(own, groups, n, hkv=1, bs=8, seed=15)
    q = b.rows(2, packed=False)
    got = run_shared(b, q, groups, n, 1, 0.1)
    check_rows(b, got, q, 0.1, decode=True)


# ------------------------------------------------------------------------------- decode

def run_decode(b, q, q_len, scale, window=0, softcap=0.0, slopes=None, num_splits=0):
    pool = b.pool()
    B = len(b.lens)
    got = pgd.paged_gqa_decode_ex(
        pool, q.view(B, q_len, -1, b.d).cuda().contiguous(), b.table.cuda(), b.len_t.cuda(),
        scale, window=window, softcap=softcap,
        slopes=None if slopes is None else slopes.cuda(), num_splits=num_splits)
    ok(pool)
    pool.close()
    return got.cpu().view(B * q_len, -1, b.d)


@pytest.mark.parametrize("q_len,window", [(1, 0), (3, 0), (2, 25)])
@pytest.mark.parametrize("shape", ["cap", "bias", "both"])
@pytest.mark.parametrize("pages,scales,d", FORMS)
def test_decode(pages, scales, d, shape, q_len, window):
    for hkv, group, bs in ((2, 3, 16), (8, 4, 8), (1, 20, 64)):
        b = Batch([1, 40, 0, 129, 33, 64, 2, 300], [q_len] * 8, hkv=hkv, d=d, bs=bs, pages=pages,
                  scales=scales, seed=bs)
        q = b.rows(hkv * group, packed=False) * 3
        kw = shape_of(shape, hkv * group)
        got = run_decode(b, q, q_len, d ** -0.5, window=window, **kw)
        check_rows(b, got, q, d ** -0.5, decode=True, window=window, **kw)


@pytest.mark.parametrize("B,hkv,group", [(1, 1, 8), (3, 8, 8), (20, 8, 4), (70, 8, 4), (2, 2, 32)])
@pytest.mark.parametrize("pages", ["bf16", "int8"])
def test_decode_long_runs(B, hkv, group, pages):
    """Runs over many spans, over two to five of them, and within one: each form of the join."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(200, 900, (B,), generator=g).tolist()
    b = Batch(lens, [1] * B, hkv=hkv, pages=pages, seed=B)
    q = b.rows(hkv * group, packed=False) * 3
    kw = dict(softcap=20.0, slopes=alibi(hkv * group))
    for splits in (0, 7, 500):
        got = run_decode(b, q, 1, 128 ** -0.5, num_splits=splits, **kw)
        check_rows(b, got, q, 128 ** -0.5, decode=True, **kw)


@pytest.mark.parametrize("B,hkv,group,q_len", [(1, 1, 8, 1), (2, 8, 4, 2), (30, 4, 3, 1),
                                               (200, 2, 2, 1)])
def test_decode_heads_of_64(B, hkv, group, q_len):
    """Joined runs, long and short, and more runs than spans, which their last arriver merges."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(2, 1200 if B < 100 else 150, (B,), generator=g).tolist()
    b = Batch(lens, [q_len] * B, hkv=hkv, d=64, seed=B)
    q = b.rows(hkv * group, packed=False) * 2
    for kw in (dict(softcap=20.0), dict(slopes=alibi(hkv * group))):
        for splits in (0, 40):
            got = run_decode(b, q, q_len, 0.125, num_splits=splits, **kw)
            check_rows(b, got, q, 0.125, decode=True, **kw)


@pytest.mark.parametrize("d", [64, 128])
def test_decode_float32(d):
    """The float32 path: 1e-5 for values and weights near 1, as for plain scores."""
    b = Batch([1, 40, 0, 129, 300], [1] * 5, hkv=2, d=d, pages="f32", seed=1)
    q = b.rows(6, packed=False)
    for kw in (dict(softcap=2.0), dict(slopes=alibi(6)), dict(softcap=30.0, slopes=alibi(6))):
        got = run_decode(b, q, 1, d ** -0.5, **kw)
        want, _ = shaped.attend(q, b.k, b.v, None, None, b.cu, b.table, b.lens, d ** -0.5, **kw)
        for r, y in want.items():
            assert (got[r].double() - y).abs().max() <= 1e-5


def test_decode_plain_arguments_are_the_plain_decode():
    """softcap 0 and no slopes: the same bits as the plain call, also by the C entry point."""
    b = Batch([40, 500, 77], [1] * 3, hkv=8, seed=2)
    pool = b.pool()
    q = b.rows(32, packed=False).view(3, 1, 32, 128).cuda()
    table, lens = b.table.cuda(), b.len_t.cuda()
    x = pgd.paged_gqa_decode(pool, q.view(3, 32, 128), table, lens, 0.1)
    y = pgd.paged_gqa_decode_ex(pool, q, table, lens, 0.1, softcap=0.0)
    assert torch.equal(x, y.view_as(x))
    pool.close()


# ---------------------------------------------------------------------- shared prefixes

def run_shared(b, q, groups, n, q_len, scale, softcap=0.0, slopes=None, status=0, **kw):
    pool = b.pool()
    B = len(b.lens)
    cu, shared = group_tables(groups, n)
    got = pgd.paged_gqa_decode_shared(
        pool, q.view(B, q_len, -1, b.d).cuda().contiguous(), cu, shared, b.table.cuda(),
        b.len_t.cuda(), scale, softcap=softcap,
        slopes=None if slopes is None else slopes.cuda(), **kw)
    assert pgd.paged_gqa_get_error(pool) == status
    pool.close()
    return got.cpu().view(B * q_len, -1, b.d)


@pytest.mark.parametrize("q_len", [1, 3])
@pytest.mark.parametrize("shape", ["plain", "cap", "both"])
@pytest.mark.parametrize("pages,scales,d", FORMS)
def test_shared(pages, scales, d, shape, q_len):
    """Prefixes that end inside blocks, of a few tokens and of none, a group of one, sequences
    without tokens, sequences of no group, own parts of one token and more."""
    groups, n = [(1, 5), (5, 6), (6, 9), (9, 11)], [300, 77, 0, 37]
    own = [50, 3, 140, -1, 20, 9, 33, 64, 5, 3, 4, 120]
    for hkv, group, bs in ((2, 3, 16), (8, 2, 32), (1, 20, 8)):
        b = shared_batch(own, groups, n, q_len, hkv=hkv, d=d, bs=bs, pages=pages, scales=scales,
                         seed=bs)
        q = b.rows(hkv * group, packed=False) * 2
        kw = {} if shape == "plain" else shape_of(shape, hkv * group)
        got = run_shared(b, q, groups, n, q_len, d ** -0.5, **kw)
        check_rows(b, got, q, d ** -0.5, decode=True, **kw)
        if q_len == 1:
            assert torch.all(got[3] == 0)


@pytest.mark.parametrize("pages,scales", [("bf16", "head"), ("e4m3", "block")])
@pytest.mark.parametrize("B,hkv,group,prefix",
                         [(40, 1, 8, 2500), (5, 8, 4, 1300), (100, 2, 4, 600)])
def test_shared_long(B, hkv, group, prefix, pages, scales):
    """Many parts of a prefix, paired blocks of rows and more than 256 rows."""
    g = torch.Generator().manual_seed(B)
    own = torch.randint(1, 100, (B,), generator=g).tolist()
    groups, n = [(0, B)], [prefix]
    b = shared_batch(own, groups, n, hkv=hkv, pages=pages, scales=scales, seed=B)
    q = b.rows(hkv * group, packed=False) * 2
    for kw in ({}, dict(softcap=10.0), dict(slopes=alibi(hkv * group))):
        got = run_shared(b, q, groups, n, 1, 128 ** -0.5, **kw)
        check_rows(b, got, q, 128 ** -0.5, decode=True, **kw)


def test_shared_lengths_beyond_what_is_seen():
    """A shared length beyond the shortest sequence of the group counts only as far as every
    query sees; all sequences the same whole length; a length of 2^31 - 1."""
    groups = [(0, 3), (3, 5), (5, 7)]
    own = [0, 0, 0, 0, 0, 40, 1]
    b = shared_batch(own, groups, [96, 37, 100], 2, hkv=2, seed=3)
    q = b.rows(8, packed=False)
    for n in ([96, 37, 100], [2 ** 31 - 1, 38, 101], [500, 2 ** 31 - 1, 100]):
        got = run_shared(b, q, groups, n, 2, 0.1)
        check_rows(b, got, q, 0.1)


@pytest.mark.parametrize("bad", ["descending", "beyond", "negative", "below"])
def test_shared_impossible_groups(bad):
    """Reported, and every sequence is read whole."""
    groups, n = [(0, 3), (3, 6)], [64, 32]
    b = shared_batch([10, 20, 30, 5, 6, 7], groups, n, hkv=2, seed=4)
    q = b.rows(4, packed=False)
    pool = b.pool()
    cu, shared = group_tables(groups, n)
    if bad == "descending":
        cu[1], cu[2] = 6, 3
    elif bad == "beyond":
        cu[2] = 7
    elif bad == "negative":
        shared[1] = -1
    else:
        cu[0] = -2
    got = pgd.paged_gqa_decode_shared(pool, q.cuda(), cu, shared, b.table.cuda(), b.len_t.cuda(),
                                      0.1)
    assert pgd.paged_gqa_get_error(pool) == _lib.PGD_ERR_SEQ_LEN
    check_rows(b, got.cpu(), q, 0.1)
    pool.close()


def test_shared_bad_blocks_and_lengths():
    """A block id out of range in a prefix: the group's rows are NaN; in a sequence's own part:
    its rows; a length out of range: its rows.  The others are right."""
    groups, n = [(0, 3), (3, 6)], [200, 300]
    b = shared_batch([10, 20, 30, 5, 6, 7], groups, n, hkv=2, seed=4)
    q = b.rows(4, packed=False)
    want, size = shaped.attend(q, b.k, b.v, None, None, b.cu, b.table, b.lens, 0.1)
    for row, col, lost in ((0, 5, {0, 1, 2}), (4, 19, {4}), (None, None, {4})):
        pool = b.pool()
        cu, shared = group_tables(groups, n)
        table, lens = b.table.cuda(), b.len_t.cuda()
        if row is None:
            lens[4] = table.shape[1] * 16 + 1
        else:
            table[row, col] = b.k.shape[0] + 5
        got = pgd.paged_gqa_decode_shared(pool, q.cuda(), cu, shared, table, lens, 0.1).cpu()
        assert pgd.paged_gqa_get_error(pool) == (
            _lib.PGD_ERR_SEQ_LEN if row is None else _lib.PGD_ERR_BLOCK_ID)
        for r, y in want.items():
            if r in lost:
                assert torch.all(got[r].isnan())
            else:
                tol = 2.0 ** -8 * y.abs() + (2.0 ** -8 + 2.0 ** -12) * size[r]
                assert torch.all((got[r].double() - y).abs() <= tol)
        pool.close()


def test_shared_without_groups():
    """No group at all is the plain decode; so is a batch of no sequences."""
    b = Batch([40, 129, 0], [1] * 3, hkv=2, seed=5)
    q = b.rows(4, packed=False)
    pool = b.pool()
    empty = torch.zeros(0, dtype=torch.int32, device="cuda")
    got = pgd.paged_gqa_decode_shared(pool, q.cuda(), torch.zeros(1, dtype=torch.int32,
                                                                  device="cuda"), empty,
                                      b.table.cuda(), b.len_t.cuda(), 0.1)
    ok(pool)
    check_rows(b, got.cpu(), q, 0.1)
    none = pgd.paged_gqa_decode_shared(pool, q[:0].cuda(), empty.new_zeros(1), empty,
                                       b.table[:0].cuda(), b.len_t[:0].cuda(), 0.1)
    assert none.shape == (0, 4, 128)
    pool.close()


def test_workspaces_are_left_ready():
    """One workspace for many steps of different lengths: each is right, and the same bits as
    with a fresh one."""
    groups, n = [(0, 4)], [150]
    b = shared_batch([1, 60, 30, 200], groups, n, hkv=2, seed=6)
    q = b.rows(8, packed=False)
    pool = b.pool()
    ws = pgd.alloc_workspace_shared(pool, 4, 1, 8, 1)
    cu, shared = group_tables(groups, n)
    lens = b.len_t.clone()
    for step in range(5):
        args = (q.cuda(), cu, shared, b.table.cuda(), lens.cuda(), 0.1)
        x = pgd.paged_gqa_decode_shared(pool, *args, workspace=ws)
        y = pgd.paged_gqa_decode_shared(pool, *args)
        ok(pool)
        assert torch.equal(x, y)
        b.lens = lens.tolist()
        check_rows(b, x.cpu(), q, 0.1)
        lens -= torch.tensor([0, 11, 3, 40])
    pool.close()


# ------------------------------------------------------------- streams, graphs, refusals

def test_captured_and_replayed():
    """The three operators captured into one graph, replayed on other inputs and lengths."""
    groups, n = [(0, 3)], [130]
    b = shared_batch([20, 7, 64], groups, n, hkv=2, seed=7)
    q = b.rows(4, packed=False)
    pool = b.pool()
    dq, table, lens = q.cuda(), b.table.cuda(), b.len_t.cuda()
    cu = b.cu.cuda()
    cg, shared = group_tables(groups, n)
    sl = alibi(4).cuda()
    vis = torch.tensor([[3, 1000]] * 3, dtype=torch.int32, device="cuda")
    ws = pgd.alloc_workspace_shared(pool, 3, 1, 4, 1)
    wd = pgd.alloc_workspace(pool, 3, 4)
    outs = [torch.zeros_like(dq) for _ in range(3)]

    def step():
        pgd.paged_gqa_attend(pool, dq, cu, table, lens, 0.1, softcap=5.0, slopes=sl, visible=vis,
                             out=outs[0])
        pgd.paged_gqa_decode_ex(pool, dq.view(3, 1, 4, 128), table, lens, 0.1, softcap=5.0,
                                slopes=sl, workspace=wd, out=outs[1].view(3, 1, 4, 128))
        pgd.paged_gqa_decode_shared(pool, dq, cg, shared, table, lens, 0.1, softcap=5.0,
                                    slopes=sl, workspace=ws, out=outs[2])

    step()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        step()
    for turn in range(3):
        q = q.roll(1, 0)
        dq.copy_(q)
        lens.copy_(b.len_t - turn)
        b.lens = (b.len_t - turn).tolist()
        graph.replay()
        torch.cuda.synchronize()
        ok(pool)
        kw = dict(softcap=5.0, slopes=sl.cpu())
        check_rows(b, outs[0].cpu(), q, 0.1, visible=vis.cpu(), **kw)
        check_rows(b, outs[1].cpu(), q, 0.1, **kw)
        check_rows(b, outs[2].cpu(), q, 0.1, **kw)
    pool.close()


def test_two_streams():
    """Calls on two streams at once, with workspaces of their own."""
    groups, n = [(0, 6)], [700]
    b = shared_batch([20, 7, 64, 1, 90, 33], groups, n, hkv=2, seed=8)
    q = b.rows(8, packed=False)
    pool = b.pool()
    dq, table, lens = q.cuda(), b.table.cuda(), b.len_t.cuda()
    cg, shared = group_tables(groups, n)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [pgd.alloc_workspace_shared(pool, 6, 1, 8, 1) for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            outs[i].append(pgd.paged_gqa_decode_shared(pool, dq, cg, shared, table, lens, 0.1,
                                                       workspace=ws[i], stream=s))
    torch.cuda.synchronize()
    ok(pool)
    check_rows(b, outs[0][0].cpu(), q, 0.1)
    for x in outs[0] + outs[1]:
        assert torch.equal(x, outs[0][0])
    pool.close()


def test_refusals():
    """Argument errors are raised before anything is launched."""
    b = Batch([40, 30], [1, 1], hkv=2, seed=9)
    pool = b.pool()
    q = b.rows(4, packed=False).cuda()
    cu, table, lens = b.where()
    cg = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    shared = torch.tensor([16], dtype=torch.int32, device="cuda")
    q4 = q.view(2, 1, 4, 128)

    def calls(**kw):
        yield lambda: pgd.paged_gqa_attend(pool, q, cu, table, lens, 0.1, **kw)
        yield lambda: pgd.paged_gqa_decode_ex(pool, q4, table, lens, 0.1, **kw)
        yield lambda: pgd.paged_gqa_decode_shared(pool, q, cg, shared, table, lens, 0.1, **kw)

    for cap in (-1.0, float("nan"), float("inf"), 2.0 ** -70, 2.0 ** 70):
        for call in calls(softcap=cap):
            with pytest.raises(pgd.PagedGQAError, match="PGD_ERR_ARG"):
                call()
    for sl, err in ((torch.ones(3), ValueError), (torch.ones(4).double(), TypeError)):
        for call in calls(slopes=sl.cuda()):
            with pytest.raises(err):
                call()
    for call in calls(slopes=torch.ones(4)):
        with pytest.raises(ValueError):
            call()
    for vis, err in ((torch.zeros(2, 3, dtype=torch.int32), ValueError),
                     (torch.zeros(3, 2, dtype=torch.int32), ValueError),
                     (torch.zeros(2, 2), TypeError)):
        with pytest.raises(err):
            pgd.paged_gqa_attend(pool, q, cu, table, lens, 0.1, visible=vis.cuda())
    odd = torch.zeros(5, dtype=torch.int32, device="cuda")[1:].view(2, 2)
    with pytest.raises(pgd.PagedGQAError, match="PGD_ERR_ALIGN"):
        pgd.paged_gqa_attend(pool, q, cu, table, lens, 0.1, visible=odd)
    with pytest.raises(pgd.PagedGQAError, match="PGD_ERR_ARG"):
        pgd.paged_gqa_decode_shared(pool, q, cg, shared, table, lens, float("inf"))
    with pytest.raises(pgd.PagedGQAError, match="PGD_ERR_ARG"):
        pgd.paged_gqa_decode_shared(pool, q, cg, shared, table, lens, 0.1, out=q)
    small = torch.zeros(pgd.paged_gqa_workspace_size_shared(pool, 2, 1, 4, 1) - 1,
                        dtype=torch.uint8, device="cuda")
    with pytest.raises(pgd.PagedGQAError, match="PGD_ERR_WORKSPACE"):
        pgd.paged_gqa_decode_shared(pool, q, cg, shared, table, lens, 0.1, workspace=small)
    with pytest.raises(pgd.PagedGQAError, match="PGD_ERR_SHAPE"):
        pgd.paged_gqa_decode_shared(pool, q.repeat(1, 40, 1), cg, shared, table, lens, 0.1)
    ok(pool)
    pool.close()
    b = Batch([40, 30], [1, 1], hkv=2, pages="f32", seed=9)
    pool = b.pool()
    q = b.rows(4, packed=False).cuda()
    with pytest.raises(pgd.PagedGQAError, match="PGD_ERR_UNSUPPORTED"):
        pgd.paged_gqa_decode_shared(pool, q, cg, shared, table, lens, 0.1)
    with pytest.raises(pgd.PagedGQAError, match="PGD_ERR_UNSUPPORTED"):
        pgd.paged_gqa_attend(pool, q, cu, table, lens, 0.1, softcap=1.0)
    pool.close()


@pytest.mark.parametrize("pages", ["bf16", "e4m3"])
def test_a_prompt_and_its_samples(pages):
    """As the operators are used together: a capped prompt is written and attends to itself,
    the block manager forks it, and every sample takes capped steps over the shared prefix;
    decode of each sequence alone gives the same answers."""
    prompt, samples, bs, hkv, hq, steps, cap = 83, 4, 16, 2, 8, 5, 6.0
    blocks = 40
    b = Batch([prompt], [prompt], hkv=hkv, bs=bs, pages=pages, scales="block", seed=10,
              spare=blocks - -(-prompt // bs))
    kvm = pgd.KVBlockManager(blocks, bs, max_seqs=samples, max_blocks_per_seq=blocks)
    pool = b.pool()
    kvm.add_sequence(0)
    for _ in range(prompt):
        kvm.append_slots([0])
    table, lens = [torch.from_numpy(x).cuda() for x in kvm.block_tables([0])]
    g = torch.Generator().manual_seed(1)
    new = lambda n, h: torch.randn(n, h, 128, generator=g).to(torch.bfloat16).cuda()
    cu = torch.tensor([0, prompt], dtype=torch.int32, device="cuda")
    q, k, v = new(prompt, hq), new(prompt, hkv), new(prompt, hkv)
    pgd.paged_kv_write(pool, k, v, cu, table, lens)
    out = pgd.paged_gqa_attend(pool, q, cu, table, lens, 0.2, softcap=cap)
    ok(pool)
    b.table, b.lens, b.cu = table.cpu(), [prompt], cu.cpu()
    take = lambda: [setattr(b, x, y.cpu()) for x, y in (
        ("k", b.dk), ("v", b.dv), ("k_scale", b.dks), ("v_scale", b.dvs)) if y is not None]
    take()
    check_rows(b, out.cpu(), q.cpu(), 0.2, softcap=cap)
    for s in range(1, samples):
        kvm.fork(0, s)
    ids = list(range(samples))
    one = torch.arange(samples + 1, dtype=torch.int32, device="cuda")
    cg = torch.tensor([0, samples], dtype=torch.int32, device="cuda")
    # 8-bit pages with block scales: a copied block is coded again as it fills, so what the
    # samples share to the bit are the prompt's whole blocks
    shared = torch.tensor([prompt // bs * bs], dtype=torch.int32, device="cuda")
    ws = pgd.alloc_workspace_shared(pool, samples, 1, hq, 1)
    for _ in range(steps):
        slots, copies = kvm.append_slots(ids)
        if copies:
            src, dst = (torch.tensor(c, dtype=torch.int32, device="cuda") for c in zip(*copies))
            pgd.paged_kv_copy_blocks(pool, src, dst)
        table, lens = [torch.from_numpy(x).cuda() for x in kvm.block_tables(ids)]
        q, k, v = new(samples, hq), new(samples, hkv), new(samples, hkv)
        pgd.paged_kv_write(pool, k, v, one, table, lens)
        out = pgd.paged_gqa_decode_shared(pool, q, cg, shared, table, lens, 0.2, softcap=cap,
                                          workspace=ws)
        alone = pgd.paged_gqa_decode_ex(pool, q.view(samples, 1, hq, 128), table, lens, 0.2,
                                        softcap=cap)
        ok(pool)
        b.table, b.lens, b.cu = table.cpu(), lens.tolist(), one.cpu()
        take()
        check_rows(b, out.cpu(), q.cpu(), 0.2, decode=True, softcap=cap)
        check_rows(b, alone.cpu().view_as(out), q.cpu(), 0.2, decode=True, softcap=cap)
    pool.close()
