"""Attention with shaped scores, decode and shared prefixes where they can go wrong: blocks of
rows without a tile, steep and far biases, small values under a cap, workspaces of many shapes,
given streams, the C entry points."""
import pytest
import torch

import paged_gqa_decode_04_gb300 as pgd
from oracle import shaped
from page_ops_cases import Batch
from paged_gqa_decode_04_gb300 import _lib
from shaped_cases import alibi, check_rows, group_tables, shared_batch, tail

pytestmark = pytest.mark.gpu


def ok(pool):
    assert pgd.paged_gqa_get_error(pool) == 0


def busy(n=1 << 26):
    """A stream that reads and writes memory without a pause, as a call's neighbour."""
    s = torch.cuda.Stream()
    x = torch.zeros(n, device="cuda")
    torch.cuda.synchronize()

    def work():
        with torch.cuda.stream(s):
            for _ in range(3):
                x.add_(1.0)
    return work


def check_again_and_again(b, heads, times=40, **kw):
    """The call many times over on two streams beside other work: the first result against the
    definition, every other one the same bits."""
    q = b.rows(heads) * 3
    scale = b.d ** -0.5
    pool, dq, where = b.pool(), b.to(q), b.where()
    dev = {k: v.cuda() if torch.is_tensor(v) else v for k, v in kw.items()}
    outs = [torch.full((b.total, heads, b.d), 7.0, dtype=b.act, device="cuda")
            for _ in range(times)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    work = busy()
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        work()
        pgd.paged_gqa_attend(pool, dq, *where, scale, out=out, stream=streams[i % 2], **dev)
    torch.cuda.synchronize()
    ok(pool)
    pool.close()
    first = outs[0].cpu()
    check_rows(b, first, q, scale, **kw)
    assert torch.all(first[int(b.cu[-1]):] == 7)
    for out in outs:
        assert torch.equal(out, outs[0])
    return first


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hide", [(0, 128), (100, 500), (200, 600), (472, 600)])
def test_blocks_of_rows_that_see_nothing(hide, d):
    """Hidden rows that fill blocks of 128 (32 tokens of 4 heads a group) at the beginning, inside
    and at the end of a sequence, beside blocks that see something."""
    b = Batch([600, 40], [600, 40], hkv=2, d=d, seed=hide[0], pad=2)
    vis = torch.tensor([[0, 2 ** 31 - 1]], dtype=torch.int32).repeat(b.total, 1)
    vis[hide[0]:hide[1], 1] = 0
    for kw in ({}, dict(softcap=20.0), dict(softcap=100.0), dict(slopes=alibi(8))):
        got = check_again_and_again(b, 8, visible=vis, **kw)
        assert torch.all(got[hide[0]:hide[1]] == 0)


@pytest.mark.parametrize("d", [64, 128])
def test_cross_attention_to_nothing(d):
    """Sequences without cached tokens beside one with many, every query of theirs zeros."""
    b = Batch([0, 300, 0], [200, 100, 33], hkv=2, d=d, seed=1)
    for kw in (dict(softcap=20.0), dict(slopes=alibi(8))):
        got = check_again_and_again(b, 8, causal=False, **kw)
        assert torch.all(got[:200] == 0) and torch.all(got[300:] == 0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [1, 20, 200])
def test_short_sequences_in_wide_clusters(rows, d):
    """Sequences of one to three tiles behind a table for 512, whose width is what the cluster size
    is chosen by: CTAs of a cluster without a tile, in calls of few and of many rows."""
    b = Batch([max(rows, x) for x in (30, 128, 300, 1)], [rows, rows, rows, min(rows, 2)], hkv=1,
              d=d, seed=rows)
    wide = torch.full((4, 4096 - b.table.shape[1]), -1, dtype=torch.int32)
    b.table = torch.cat([b.table, wide], 1).contiguous()
    vis = torch.tensor([[0, 2 ** 31 - 1]], dtype=torch.int32).repeat(b.total, 1)
    vis[::3, 1] = 10
    for kw in (dict(softcap=20.0), dict(slopes=alibi(4)), dict(visible=vis)):
        check_again_and_again(b, 4, **kw)


@pytest.mark.parametrize("d", [64, 128])
def test_sequences_of_impossible_length(d):
    """Their rows are NaN, not what lay in shared memory; the others are right."""
    b = Batch([200, 70], [200, 70], hkv=2, d=d, seed=2)
    q = b.rows(8)
    pool, dq = b.pool(), b.to(q)
    cu, table, lens = b.where()
    lens[0] = table.shape[1] * b.bs + 1
    work = busy()
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        work()
        outs.append(pgd.paged_gqa_attend(pool, dq, cu, table, lens, 0.1, softcap=20.0))
    torch.cuda.synchronize()
    assert pgd.paged_gqa_get_error(pool) == _lib.PGD_ERR_SEQ_LEN
    pool.close()
    want, size = shaped.attend(q, b.k, b.v, None, None, b.cu, b.table, b.lens, 0.1, softcap=20.0)
    for out in outs:
        assert torch.all(out[:200].isnan()) and torch.equal(out[200:], outs[0][200:])
    for row in range(200, 270):
        tol = 2.0 ** -8 * want[row].abs() + (2.0 ** -8 + 2.0 ** -12) * size[row]
        assert torch.all((outs[0][row].cpu().double() - want[row]).abs() <= tol)


@pytest.mark.parametrize("as_int", [False, True])
def test_decodes_on_a_given_stream_without_a_workspace(as_int):
    """Decodes make their workspace and output on the stream that they are launched on: with
    the current stream busy, and its memory dirty and soon handed out again, every result is
    right."""
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(500, 4000, (6,), generator=g).tolist()
    b = Batch(lens, [1] * 6, hkv=2, d=64, seed=6)
    q = b.rows(8, packed=False)
    pool, dq, table, lens = b.pool(), q.cuda(), b.table.cuda(), b.len_t.cuda()
    h_q, h_table, h_lens = q.contiguous(), b.table, b.len_t
    n = max(pgd.paged_gqa_workspace_size_host(pool, 6, 1, 8, b.table.shape[1]), 1 << 20)
    side = torch.cuda.Stream()
    x = torch.zeros(1 << 26, device="cuda")
    torch.cuda.synchronize()
    outs, host, s = [], [], side.cuda_stream if as_int else side
    for i in range(30):
        for _ in range(2):
            x.add_(1.0)
        dirt = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        del dirt
        kw = dict(softcap=20.0) if i % 3 == 0 else {}
        if i % 3 < 2:
            outs.append((kw, pgd.paged_gqa_decode_ex(pool, dq.view(6, 1, 8, 64), table, lens, 0.1,
                                                     stream=s, **kw)))
        else:
            outs.append((kw, pgd.paged_gqa_decode(pool, dq, table, lens, 0.1, stream=s)))
        host.append(pgd.paged_gqa_decode_host(pool, h_q, h_table, h_lens, 0.1, stream=s))
        dirt = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        del dirt
    torch.cuda.synchronize()
    ok(pool)
    for i, (kw, out) in enumerate(outs):
        got = out.cpu().view(6, 8, 64)
        if i < 3:
            check_rows(b, got, q, 0.1, decode=True, **kw)
        assert torch.equal(got, outs[i % 3 if kw else 1][1].cpu().view(6, 8, 64))
        assert torch.equal(host[i], outs[1][1].cpu().view(6, 8, 64))
    pool.close()


def test_decodes_refuse_outputs_and_workspaces():
    """Raised before anything is launched; a larger output and a workspace of another type are
    fine."""
    b = Batch([40, 30], [1, 1], hkv=2, seed=9)
    pool, q = b.pool(), b.rows(4, packed=False)
    dq, table, lens = q.cuda(), b.table.cuda(), b.len_t.cuda()
    n = pgd.paged_gqa_workspace_size_host(pool, 2, 1, 4, table.shape[1])
    out = torch.full((3, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")

    def calls(**kw):
        yield lambda: pgd.paged_gqa_decode(pool, dq, table, lens, 0.1, **kw)
        yield lambda: pgd.paged_gqa_decode_ex(pool, dq.view(2, 1, 4, 128), table, lens, 0.1, **kw)

    for kw, err in ((dict(out=out.cpu()), ValueError), (dict(out=out[:1]), ValueError),
                    (dict(out=out.float()), TypeError), (dict(workspace=ws.cpu()), ValueError),
                    (dict(workspace=torch.zeros(2 * n, dtype=torch.uint8, device="cuda")[::2]),
                     ValueError)):
        for call in calls(**kw):
            with pytest.raises(err):
                call()
    for bad in (ws.cpu(), torch.zeros(2 * n, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            pgd.paged_gqa_decode_host(pool, q.contiguous(), b.table, b.len_t, 0.1, workspace=bad)
    words = torch.zeros(-(-n // 4), dtype=torch.int32, device="cuda")
    for call in calls(out=out, workspace=words):
        call()
        torch.cuda.synchronize()
        ok(pool)
        check_rows(b, out.cpu(), q, 0.1, decode=True)
        assert torch.all(out[2] == 7)
        out[:2] = 0
    pool.close()


# Slopes whose bias is beyond float32 at the distances of a test, on both sides of the one from
# which on they count alike, and an ordinary one.  Raw scores differ by far less than 2^13, so
# that all but the last leave one token, the nearest or the farthest.
STEEP = torch.tensor([3.4e38, -1e30, 2.0 ** 25, -2.0 ** 20, 9000.0, 1.0])


@pytest.mark.parametrize("pages,scales,d", [("f32", "head", 128), ("f32", "head", 64),
                                            ("bf16", "head", 64), ("bf16", "head", 128),
                                            ("e4m3", "head", 128), ("e4m3", "block", 128),
                                            ("int8", "head", 128), ("int8", "block", 128)])
def test_decode_steep_slopes(pages, scales, d):
    b = Batch([1, 300, 40, 1200], [1] * 4, hkv=2, d=d, pages=pages, scales=scales, seed=1)
    q = b.rows(6, packed=False)
    pool = b.pool()
    for cap in (0.0, 20.0):
        got = pgd.paged_gqa_decode_ex(pool, q.view(4, 1, 6, d).cuda(), b.table.cuda(),
                                      b.len_t.cuda(), 0.1, softcap=cap, slopes=STEEP.cuda())
        ok(pool)
        got = got.cpu().view(4, 6, d)
        if pages != "f32":
            check_rows(b, got, q, 0.1, decode=True, softcap=cap, slopes=STEEP)
            continue
        want, _ = shaped.attend(q, b.k, b.v, None, None, b.cu, b.table, b.lens, 0.1, softcap=cap,
                                slopes=STEEP)
        for r, y in want.items():
            assert (got[r].double() - y).abs().max() <= 1e-5
    pool.close()


@pytest.mark.parametrize("pages,scales", [("bf16", "head"), ("e4m3", "head"), ("e4m3", "block"),
                                          ("int8", "head"), ("int8", "block")])
def test_attend_steep_slopes(pages, scales):
    b = Batch([300, 140], [130, 140], hkv=2, pages=pages, scales=scales, seed=2)
    q = b.rows(6)
    pool, dq, where = b.pool(), b.to(q), b.where()
    for causal in (True, False):
        for cap in (0.0, 20.0):
            got = pgd.paged_gqa_attend(pool, dq, *where, 0.1, causal=causal, softcap=cap,
                                       slopes=STEEP.cuda()).cpu()
            ok(pool)
            check_rows(b, got, q, 0.1, causal=causal, softcap=cap, slopes=STEEP)
    pool.close()


@pytest.mark.parametrize("pages,scales", [("bf16", "head"), ("e4m3", "head"), ("e4m3", "block"),
                                          ("int8", "head")])
@pytest.mark.parametrize("causal", [True, False])
def test_attend_bias_of_what_is_far_away(pages, scales, causal):
    """Rows that see only tokens far behind, far ahead or on one side of themselves.  Biases reach
    2^25 in units of log 2 there; what is left of them among the tokens a row sees is below 2^21
    at the slopes where one token is left, and below 2^10 at the others."""
    b = Batch([3000, 200], [3000, 200], hkv=1, pages=pages, scales=scales, seed=3)
    vis = torch.zeros(b.total, 2, dtype=torch.int32)
    vis[0::4] = torch.tensor([0, 100])
    vis[1::4] = torch.tensor([2900, 3000])
    vis[2::4] = torch.tensor([1400, 1500])
    vis[3::64] = torch.tensor([1490, 1500])
    slopes = torch.cat([STEEP, alibi(2)])
    q = b.rows(8)
    pool, dq, where = b.pool(), b.to(q), b.where()
    got = pgd.paged_gqa_attend(pool, dq, *where, 0.1, causal=causal, slopes=slopes.cuda(),
                               visible=vis.cuda()).cpu()
    ok(pool)
    pool.close()
    check_rows(b, got, q, 0.1, causal=causal, slopes=slopes, visible=vis)


@pytest.mark.parametrize("pages,scales", [("bf16", "head"), ("e4m3", "head"), ("e4m3", "block"),
                                          ("int8", "head")])
@pytest.mark.parametrize("causal", [True, False])
def test_attend_bias_of_what_is_very_far_away(pages, scales, causal):
    """The same at the end of a long sequence, where whole biases reach 2^29 in units of log 2:
    steps of 32, beyond what an f16 weight can hold."""
    b = Batch([40000], [40], hkv=1, pages=pages, scales=scales, seed=5)
    vis = torch.zeros(40, 2, dtype=torch.int32)
    vis[0::2] = torch.tensor([0, 300])
    vis[1::2] = torch.tensor([64, 1000])
    slopes = torch.cat([STEEP, alibi(2)])
    q = b.rows(8)
    pool, dq, where = b.pool(), b.to(q), b.where()
    got = pgd.paged_gqa_attend(pool, dq, *where, 0.1, causal=causal, slopes=slopes.cuda(),
                               visible=vis.cuda()).cpu()
    ok(pool)
    pool.close()
    check_rows(b, got, q, 0.1, causal=causal, slopes=slopes, visible=vis)


@pytest.mark.parametrize("pages,scales", [("bf16", "head"), ("e4m3", "head"), ("int8", "block")])
@pytest.mark.parametrize("q_len", [1, 3])
def test_shared_prefix_with_steep_slopes(q_len, pages, scales):
    """A prefix and own tokens whose biases differ by up to 2^24: joined by what they come to."""
    groups, n = [(0, 3), (3, 5)], [1500, 77]
    b = shared_batch([900, 3, 40, 5, 700], groups, n, q_len, hkv=2, pages=pages, scales=scales,
                     seed=4)
    slopes = torch.cat([STEEP, alibi(2)])
    q = b.rows(8, packed=False)
    pool = b.pool()
    cu, shared = group_tables(groups, n)
    for cap in (0.0, 20.0):
        got = pgd.paged_gqa_decode_shared(pool, q.view(5, q_len, 8, 128).cuda(), cu, shared,
                                          b.table.cuda(), b.len_t.cuda(), 0.1, softcap=cap,
                                          slopes=slopes.cuda())
        ok(pool)
        check_rows(b, got.cpu().view(5 * q_len, 8, 128), q, 0.1, decode=True, softcap=cap,
                   slopes=slopes)
    pool.close()


def check_rows_f16(b, got, q, scale, low, **kw):
    """The definition's rows, to the output's rounding, 2^-8, and weights of f16, 2^-11; 2^-12 for
    the rest and `low` a token for f16 below its normal numbers, as in check_rows."""
    want, size = shaped.attend(q, b.k, b.v, b.k_scale, b.v_scale, b.cu, b.table, b.lens, scale,
                               **kw)
    for row, y in want.items():
        tol = 2.0 ** -8 * y.abs() + (2.0 ** -11 + 2.0 ** -12) * size[row] + low * max(b.lens)
        err = (got[row].double() - y).abs()
        assert torch.all(err <= tol), (row, float((err - tol).max()))


@pytest.mark.parametrize("cap", [2.0, 30.0, 50.0, 60.0])
@pytest.mark.parametrize("pages,scales", [("e4m3", "head"), ("int8", "head"), ("e4m3", "block")])
def test_capped_weights_over_8_bit_pages_keep_f16(pages, scales, cap):
    """As without a cap: weights of 11 bits in the attention and in a shared prefix."""
    b = Batch([300, 160], [100, 160], hkv=2, pages=pages, scales=scales, seed=7)
    q = b.rows(6) * 3
    pool = b.pool()
    got = pgd.paged_gqa_attend(pool, b.to(q), *b.where(), 0.1, softcap=cap).cpu()
    ok(pool)
    pool.close()
    check_rows_f16(b, got, q, 0.1, tail(b, False), softcap=cap)
    groups, n = [(0, 4)], [512]
    b = shared_batch([1, 30, 100, 7], groups, n, hkv=2, pages=pages, scales=scales, seed=8)
    q = b.rows(6, packed=False) * 3
    pool = b.pool()
    cu, shared = group_tables(groups, n)
    got = pgd.paged_gqa_decode_shared(pool, q.cuda(), cu, shared, b.table.cuda(), b.len_t.cuda(),
                                      0.1, softcap=cap).cpu()
    ok(pool)
    pool.close()
    check_rows_f16(b, got, q, 0.1, tail(b, True), softcap=cap)


SIZES = [3, 40, 2, 64, 17, 64, 1, 33, 64]


@pytest.mark.parametrize("pages,scales,d,heads", [("bf16", "head", 64, (2, 8)),
                                                  ("bf16", "head", 128, (2, 8)),
                                                  ("bf16", "head", 128, (1, 20)),
                                                  ("bf16", "head", 128, (8, 64)),
                                                  ("e4m3", "block", 128, (8, 64)),
                                                  ("f32", "head", 128, (2, 8))])
def test_one_workspace_for_batches_of_any_size(pages, scales, d, heads):
    """A workspace sized for the largest batch, used by smaller and larger ones in turn, by plain
    and shaped decodes and by the one with host buffers: the bits of a fresh workspace."""
    hkv, hq = heads
    g = torch.Generator().manual_seed(d + hq)
    lens = torch.randint(100, 3000, (64,), generator=g).tolist()
    b = Batch(lens, [1] * 64, hkv=hkv, d=d, pages=pages, scales=scales, seed=3)
    q = b.rows(hq, packed=False).contiguous()
    pool = b.pool()
    dq, table, lens = q.cuda(), b.table.cuda(), b.len_t.cuda()
    ws = pgd.alloc_workspace(pool, 64, hq)
    n = pgd.paged_gqa_workspace_size_host(pool, 64, 1, hq, table.shape[1])
    wh = torch.zeros(n, dtype=torch.uint8, device="cuda")
    for B in SIZES:
        for cap in (0.0, 15.0):
            args = (pool, dq[:B].view(B, 1, hq, d), table[:B], lens[:B], 0.1)
            out = torch.full((B, 1, hq, d), 7.0, dtype=b.act, device="cuda")
            pgd.paged_gqa_decode_ex(*args, softcap=cap, out=out, workspace=ws)
            assert torch.equal(out, pgd.paged_gqa_decode_ex(*args, softcap=cap)), (B, cap)
        got = pgd.paged_gqa_decode_host(pool, q[:B], b.table[:B], b.len_t[:B], 0.1, workspace=wh)
        want = pgd.paged_gqa_decode_host(pool, q[:B], b.table[:B], b.len_t[:B], 0.1)
        torch.cuda.synchronize()
        assert torch.equal(got, want), B
    ok(pool)
    pool.close()


def test_one_workspace_for_shared_and_whole_decodes():
    """A shared decode's workspace serves decodes of its batch or fewer sequences besides."""
    g = torch.Generator().manual_seed(1)
    own = torch.randint(100, 900, (64,), generator=g).tolist()
    b = shared_batch(own, [(0, 64)], [700], hkv=2, d=64, seed=4)
    q = b.rows(8, packed=False)
    pool = b.pool()
    dq, table, lens = q.cuda(), b.table.cuda(), b.len_t.cuda()
    n = torch.tensor([700], dtype=torch.int32, device="cuda")
    ws = pgd.alloc_workspace_shared(pool, 64, 1, 8, 1)
    for B in SIZES:
        cu = torch.tensor([0, B], dtype=torch.int32, device="cuda")
        args = (pool, dq[:B], cu, n, table[:B], lens[:B], 0.1)
        x = pgd.paged_gqa_decode_shared(*args, workspace=ws)
        assert torch.equal(x, pgd.paged_gqa_decode_shared(*args)), B
        for size in (B, 64):
            args = (pool, dq[:size].view(size, 1, 8, 64), table[:size], lens[:size], 0.1)
            y = pgd.paged_gqa_decode_ex(*args, slopes=alibi(8).cuda(), workspace=ws)
            assert torch.equal(y, pgd.paged_gqa_decode_ex(*args, slopes=alibi(8).cuda())), size
    ok(pool)
    pool.close()


def test_a_shared_workspace_serves_fewer_groups_and_sequences():
    """Made for 64 sequences in 16 groups, used for 1 to 16 groups of 8 to 64."""
    own = [1 + 7 * i % 50 for i in range(64)]
    b = shared_batch(own, [(0, 64)], [300], hkv=8, seed=9)
    q = b.rows(64, packed=False)
    pool = b.pool()
    dq, table, lens = q.cuda(), b.table.cuda(), b.len_t.cuda()
    ws = pgd.alloc_workspace_shared(pool, 64, 1, 64, 16)
    for B, groups in ((64, 16), (64, 1), (32, 2), (32, 1), (8, 8), (8, 1), (64, 3)):
        cu = torch.tensor([B * g // groups for g in range(groups + 1)], dtype=torch.int32)
        n = torch.full((groups,), 300, dtype=torch.int32, device="cuda")
        args = (pool, dq[:B], cu.cuda(), n, table[:B], lens[:B], 0.1)
        x = pgd.paged_gqa_decode_shared(*args, workspace=ws)
        ok(pool)
        assert torch.equal(x, pgd.paged_gqa_decode_shared(*args))
        if B == 64:
            check_rows(b, x.cpu(), q, 0.1, decode=True)
    sizes = [pgd.paged_gqa_workspace_size_shared(pool, B, 1, 64, g)
             for B in (1, 2, 8, 33, 64, 200, 1000) for g in (1, 5, 70)]
    assert sizes == sorted(sizes)
    pool.close()


@pytest.mark.parametrize("size", [1.0, 2.0 ** -18, 2.0 ** -24, 2.0 ** -30, 2.0 ** 30])
def test_values_where_all_scores_are_at_the_lower_end_of_the_cap(size):
    """Weights near 2^-100 of a fixed reference: values of any size to the bound's steps and 2^-26,
    2^-126 over the weight."""
    b = Batch([700, 130], [140, 130], hkv=1, d=64, seed=13)
    b.k[:] = torch.where(b.k.isnan(), b.k, torch.ones((), dtype=b.k.dtype))
    b.v *= size
    q = -torch.ones(b.total, 2, 64, dtype=torch.bfloat16)
    pool, where = b.pool(), b.where()
    for cap in (55.0, 30.0):
        for causal in (True, False):
            got = pgd.paged_gqa_attend(pool, q.cuda(), *where, 40.0, causal=causal,
                                       softcap=cap).cpu()
            ok(pool)
            want, most = shaped.attend(q, b.k, b.v, None, None, b.cu, b.table, b.lens, 40.0,
                                       causal=causal, softcap=cap)
            for row, y in want.items():
                tol = 2.0 ** -8 * y.abs() + (2.0 ** -8 + 2.0 ** -12) * most[row] + 2.0 ** -26
                assert torch.all((got[row].double() - y).abs() <= tol), (row, cap)
    pool.close()


@pytest.mark.parametrize("pages,scales,d", [("bf16", "head", 64), ("bf16", "head", 128),
                                            ("e4m3", "head", 128), ("int8", "block", 128)])
def test_plain_c_entry_points(pages, scales, d):
    """paged_gqa_attend and paged_gqa_decode_ex of the C interface, which the binding does not
    call, on real data: right, and the bits of the shaped ones with nothing shaped."""
    lib = _lib.load()
    b = Batch([300, 40, 0, 129], [100, 3, 0, 129], hkv=2, d=d, pages=pages, scales=scales, seed=6)
    q = b.rows(6)
    pool, dq = b.pool(), b.to(q)
    cu, table, lens = b.where()
    for causal, window in ((1, 0), (1, 33), (0, 0)):
        got, same = [torch.full((b.total, 6, d), 7.0, dtype=b.act, device="cuda")
                     for _ in range(2)]
        first = (pool.handle, dq.data_ptr(), dq.stride(0), b.total, 6, cu.data_ptr(), 4,
                 table.data_ptr(), table.shape[1], lens.data_ptr(), causal, window, 0.1)
        assert lib.paged_gqa_attend(*first, got.data_ptr(), None) == 0
        assert lib.paged_gqa_attend_shaped(*first, 0.0, None, None, same.data_ptr(), None) == 0
        torch.cuda.synchronize()
        ok(pool)
        check_rows(b, got.cpu(), q, 0.1, causal=bool(causal), window=window)
        assert torch.equal(got, same)
    for q_len, window in ((1, 0), (3, 0), (2, 50)):
        b.cu = torch.arange(5, dtype=torch.int32) * q_len
        q = torch.randn((4 * q_len, 6, d), generator=b.g).to(b.act)
        dq = q.cuda()
        n = pgd.paged_gqa_workspace_size_ex(pool, 4, q_len, 6)
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        got, same = [torch.full((4 * q_len, 6, d), 7.0, dtype=b.act, device="cuda")
                     for _ in range(2)]
        torch.cuda.synchronize()
        first = (pool.handle, dq.data_ptr(), 4, q_len, 6, table.data_ptr(), table.shape[1],
                 lens.data_ptr(), window, 0.1)
        last = (ws.data_ptr(), n, 0, None)
        assert lib.paged_gqa_decode_ex(*first, got.data_ptr(), *last) == 0
        assert lib.paged_gqa_decode_shaped(*first, 0.0, None, same.data_ptr(), *last) == 0
        torch.cuda.synchronize()
        ok(pool)
        check_rows(b, got.cpu(), q, 0.1, decode=True, window=window)
        assert torch.equal(got, same)
    pool.close()


def test_sequences_that_are_all_prefix():
    """One query a sequence, and every cached token shared: nothing is left for the decode, in
    some sequences or in any."""
    for own in ([0, 0, 0], [0, 5, 0]):
        for n in (256, 512, 320):
            b = shared_batch(own, [(0, 3)], [n], hkv=2, bs=64, seed=n)
            q = b.rows(8, packed=False)
            pool = b.pool()
            cu, shared = group_tables([(0, 3)], [n])
            for kw in ({}, dict(softcap=20.0), dict(slopes=alibi(8))):
                dev = {k: v.cuda() if torch.is_tensor(v) else v for k, v in kw.items()}
                got = pgd.paged_gqa_decode_shared(pool, q.cuda(), cu, shared, b.table.cuda(),
                                                  b.len_t.cuda(), 0.1, **dev)
                ok(pool)
                check_rows(b, got.cpu(), q, 0.1, decode=True, **kw)
            pool.close()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kw", [{}, dict(softcap=2.0), dict(softcap=50.0), dict(softcap=60.0),
                                dict(slopes=True), dict(softcap=50.0, slopes=True)])
def test_a_row_that_sees_one_token_is_its_value(kw, d):
    """To the bit, over bfloat16 pages: the one weight is 1, to which a sum off by less than 2^-13
    rounds it, and what such a sum divides is off by far less than the half step, 2^-9, that would
    leave the value."""
    kw = dict(kw, slopes=alibi(6).cuda()) if "slopes" in kw else kw
    b = Batch([300, 1, 140], [300, 1, 140], hkv=2, d=d, seed=14)
    q = b.rows(6) * 3
    pool, dq, (cu, table, lens) = b.pool(), b.to(q), b.where()
    tokens = [(s, t) for s, n in enumerate(b.lens) for t in range(n)]
    values = torch.stack([b.v[int(b.table[s][t // 16]), t % 16] for s, t in tokens])
    values = values.repeat_interleave(3, dim=1)
    at = torch.tensor([[t, t + 1] for _, t in tokens], dtype=torch.int32, device="cuda")
    for causal in (True, False):
        got = pgd.paged_gqa_attend(pool, dq, cu, table, lens, d ** -0.5, causal=causal,
                                   visible=at, **kw)
        assert torch.equal(got.cpu(), values)
    got = pgd.paged_gqa_attend(pool, dq, cu, table, lens, d ** -0.5, **kw).cpu()
    first = [0, 300, 301]
    assert torch.equal(got[first], values[first])
    ones = torch.ones(3, dtype=torch.int32, device="cuda")
    dq = q[first].contiguous().cuda()
    got = pgd.paged_gqa_decode_ex(pool, dq.view(3, 1, 6, d), table, ones, d ** -0.5, **kw)
    assert torch.equal(got.cpu().view(3, 6, d), values[first])
    ok(pool)
    pool.close()


def test_captured_batches_of_several_sizes_share_a_workspace():
    """Graphs of a whole and of a shared decode for 3, 64 and 17 sequences, captured over one
    workspace each and replayed in turn: the bits of calls with workspaces of their own."""
    g = torch.Generator().manual_seed(2)
    own = torch.randint(50, 900, (64,), generator=g).tolist()
    b = shared_batch(own, [(0, 64)], [600], hkv=2, d=64, seed=5)
    q = b.rows(8, packed=False)
    pool = b.pool()
    dq, table, lens = q.cuda(), b.table.cuda(), b.len_t.cuda()
    n = torch.tensor([600], dtype=torch.int32, device="cuda")
    wd = pgd.alloc_workspace(pool, 64, 8)
    wsh = pgd.alloc_workspace_shared(pool, 64, 1, 8, 1)
    side, graphs = torch.cuda.Stream(), []
    for B in (3, 64, 17):
        cu = torch.tensor([0, B], dtype=torch.int32, device="cuda")
        whole = (pool, dq[:B].view(B, 1, 8, 64), table[:B], lens[:B], 0.1)
        shared = (pool, dq[:B], cu, n, table[:B], lens[:B], 0.1)
        want = [pgd.paged_gqa_decode_ex(*whole), pgd.paged_gqa_decode_ex(*whole, softcap=9.0),
                pgd.paged_gqa_decode_shared(*shared, softcap=9.0)]
        outs = [torch.zeros_like(x) for x in want]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            pgd.paged_gqa_decode_ex(*whole, out=outs[0], workspace=wd)
            pgd.paged_gqa_decode_ex(*whole, softcap=9.0, out=outs[1], workspace=wd)
            pgd.paged_gqa_decode_shared(*shared, softcap=9.0, out=outs[2], workspace=wsh)
        graphs.append((graph, outs, want, cu))
    for i in (0, 1, 2, 1, 0, 0, 2, 1):
        graph, outs, want, _ = graphs[i]
        for x in outs:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(outs, want):
            assert torch.equal(x, y)
    ok(pool)
    pool.close()
