"""The ragged page operators on the GPU against their float64 definitions: quantising
write, read back, norm and rotation with the write, attention of many query tokens."""
import pytest
import torch

import paged_gqa_decode_04_gb300 as pgd
from oracle import page_ops as ref
from page_ops_cases import ROUND, Batch, bits, check_stored
from paged_gqa_decode_04_gb300 import _lib

pytestmark = pytest.mark.gpu

# lengths and new rows: one token, none, a whole prompt, a chunk that starts inside a
# block, one that ends on a block's end, one token behind a full block
LENS = [1, 40, 0, 129, 33, 64, 17, 300]
NEW = [1, 0, 0, 129, 20, 7, 1, 45]
FORMS = [("f32", "head", 64), ("f32", "head", 128), ("bf16", "head", 64), ("bf16", "head", 128),
         ("e4m3", "head", 128), ("int8", "head", 128), ("e4m3", "block", 128),
         ("int8", "block", 128)]


def ok(pool):
    assert pgd.paged_gqa_get_error(pool) == 0


@pytest.mark.parametrize("bs", [8, 16, 64, 256])
@pytest.mark.parametrize("pages,scales,d", FORMS)
def test_write(pages, scales, d, bs):
    b = Batch(LENS, NEW, hkv=3, d=d, bs=bs, pages=pages, scales=scales, seed=bs, pad=5)
    k, v = b.rows(3), b.rows(3, packed=False)
    k[b.cu[-1]:] = float("nan")                       # rows behind the last sequence
    k[0] *= 30                                        # saturates static scales
    with b_pool(b) as pool:
        pgd.paged_kv_write(pool, b.to(k), b.to(v), *b.where())
        ok(pool)
    rows = b.held_rows()
    for name, x, after, sc in (("k", k, b.dk, b.dks), ("v", v, b.dv, b.dvs)):
        want = {r: x[r].double() for r in rows}
        check_stored(b, name, want, {r: w.abs() for r, w in want.items()}, after, sc, 0.0)


class b_pool:
    def __init__(self, batch):
        self.pool = batch.pool()

    def __enter__(self):
        return self.pool

    def __exit__(self, *_):
        self.pool.close()


@pytest.mark.parametrize("scales", ["head", "block"])
@pytest.mark.parametrize("pages", ["e4m3", "int8"])
def test_write_special_values(pages, scales):
    """Zero rows, rows below the smallest scale, infinities and NaN."""
    b = Batch([16, 32, 16, 16], [16, 16, 16, 16], hkv=2, bs=16, pages=pages, scales=scales)
    k = b.rows(2)
    k[0:16] = 0
    k[16:32] = 1e-37                                  # scale below 2^-126: zeros
    k[33, 0, 5], k[34, 0, 6], k[35, 1, 7] = float("inf"), -float("inf"), float("nan")
    with b_pool(b) as pool:
        pgd.paged_kv_write(pool, b.to(k), b.to(k), *b.where())
        ok(pool)
    blk = [int(b.table[i][(b.lens[i] - 1) // 16]) for i in range(4)]
    got = b.dk.cpu()
    assert torch.all(got[blk[0]].float() == 0) and torch.all(got[blk[1]].float() == 0)
    x = got[blk[2]].float()
    top = ref.TOP[got.dtype]
    assert x[1, 0, 5] == top and x[2, 0, 6] == -top
    assert x[3, 1, 7].isnan() if pages == "e4m3" else x[3, 1, 7] == 0
    if scales == "block":
        s = b.dks.cpu()
        assert torch.all(s[blk[0]] == 0) and torch.all(s[blk[1]] == 0)
        fin = torch.where(torch.isfinite(k[32:48].double()), k[32:48].double().abs(), 0.0)
        want = fin.amax((0, 2)) / top
        assert torch.all((s[blk[2]].double() - want).abs() <= want * 2.0 ** -23)


@pytest.mark.parametrize("pages", ["e4m3", "int8"])
def test_token_by_token_keeps_the_range(pages):
    """Rows of growing size appended one at a time: every earlier token is within half
    a step of the final scale for each time the scale grew."""
    n, bs, hkv = 40, 16, 2
    b = Batch([n], [n], hkv=hkv, bs=bs, pages=pages, scales="block")
    k = (b.rows(hkv).float() * torch.linspace(0.1, 3, n)[:, None, None]).to(torch.bfloat16)
    with b_pool(b) as pool:
        dk, dt = b.to(k), b.table.cuda()
        for t in range(n):
            pgd.paged_kv_write(pool, dk[t:t + 1], dk[t:t + 1],
                               torch.tensor([0, 1], dtype=torch.int32, device="cuda"), dt,
                               torch.tensor([t + 1], dtype=torch.int32, device="cuda"))
        ok(pool)
    got, s = b.dk.cpu(), b.dks.cpu()
    top = ref.TOP[got.dtype]
    for t in range(n):
        blk, slot = ref.place(b.table, bs, 0, t)
        x = k[t].double()
        step = s[blk].double()[:, None] * (1.0 if pages == "int8" else 32.0)  # widest spacing
        grown = bs - slot                             # at most once for each later token
        assert torch.all((got[blk, slot].double() * s[blk].double()[:, None] - x).abs()
                         <= 0.5 * step * (grown + 1) * (1 + 2.0 ** -20))
        last = min(n, (t // bs + 1) * bs)
        want = k[t // bs * bs:last].double().abs().amax((0, 2)) / top
        assert torch.all((s[blk].double() - want).abs() <= want * 2.0 ** -23)


@pytest.mark.parametrize("bs", [8, 32, 256])
@pytest.mark.parametrize("pages,scales,d", FORMS)
def test_read(pages, scales, d, bs):
    b = Batch(LENS, NEW, hkv=3, d=d, bs=bs, pages=pages, scales=scales, seed=bs, pad=4)
    out = [torch.full((b.total, 3, d), 7.0, dtype=b.act, device="cuda") for _ in range(2)]
    with b_pool(b) as pool:
        got = pgd.paged_kv_read(pool, b.total, *b.where(), out=out)
        ok(pool)
        fresh = pgd.paged_kv_read(pool, int(b.cu[-1]), *b.where())
    for x, f, p, s in zip(got, fresh, (b.k, b.v), (b.k_scale, b.v_scale)):
        want = ref.read(p, s, b.cu, b.table, b.lens)
        for r, y in want.items():
            # a float32 product, then the output's rounding
            tol = (ROUND[b.act] + 2.0 ** -23) * y.abs() if s is not None else 0.0 * y
            assert torch.all((x[r].cpu().double() - y).abs() <= tol)
        assert torch.all(x[int(b.cu[-1]):] == 7)
        assert torch.equal(bits(x[:int(b.cu[-1])]), bits(f))


def run_norm_rope(b, hq, q, k, v, **kw):
    with b_pool(b) as pool:
        out = pgd.paged_qk_norm_rope_write(pool, b.to(q), b.to(k), b.to(v), *b.where(), **kw)
        ok(pool)
    return out.cpu()


# float32 arithmetic of a normed, rotated element, relative to the magnitudes that meet in
# it: a sum of 128 squares (each partial sum one rounding, at most 8 + 4 deep: 12 * 2^-24,
# halved by the root), rsqrt (2 ulp), three products and a sum: below 2^-20
F32 = 2.0 ** -20


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm,rope_dim", [("bf16", "d"), ("f32", "half"), (None, "d"),
                                           ("bf16", None), (None, None), ("k", 16)])
@pytest.mark.parametrize("pages,scales,d", FORMS)
def test_norm_rope_write(pages, scales, d, norm, rope_dim, interleaved):
    b = Batch(LENS, NEW, hkv=2, d=d, bs=16, pages=pages, scales=scales, seed=3, pad=3)
    hq = 10
    q, k, v = b.rows(hq), b.rows(2), b.rows(2)
    wt = torch.float32 if norm == "f32" else torch.bfloat16
    qw, kw = [(1 + 0.3 * torch.randn(d, generator=b.g)).to(wt) for _ in range(2)]
    qw, kw = (None if norm in (None, "k") else qw), (kw if norm else None)
    dim = {"d": d, "half": d // 2}.get(rope_dim, rope_dim)
    rope = pgd.rope_table(max(LENS), dim) if dim else None
    out = torch.full((b.total, hq, d), 7.0, dtype=b.act, device="cuda")
    got = run_norm_rope(b, hq, q, k, v, q_weight=None if qw is None else qw.cuda(),
                        k_weight=None if kw is None else kw.cuda(), eps=1e-5,
                        rope=None if rope is None else rope.cuda(), interleaved=interleaved,
                        q_out=out)
    want_k, size_k = {}, {}
    for s in range(len(LENS)):
        for row, pos in ref.rows_of(b.cu, b.lens, s):
            y, m = ref.norm_rotate(q[row], qw, 1e-5, rope, interleaved, pos)
            tol = ROUND[b.act] * y.abs() + F32 * m
            assert torch.all((got[row].double() - y).abs() <= tol), (s, pos)
            want_k[row], size_k[row] = ref.norm_rotate(k[row], kw, 1e-5, rope, interleaved, pos)
    assert torch.all(got[int(b.cu[-1]):] == 7)
    check_stored(b, "k", want_k, size_k, b.dk, b.dks, F32)
    want = {r: v[r].double() for r in want_k}
    check_stored(b, "v", want, {r: y.abs() for r, y in want.items()}, b.dv, b.dvs, 0.0)


@pytest.mark.parametrize("bs", [8, 32, 256])
@pytest.mark.parametrize("pages,hkv", [("e4m3", 9), ("int8", 1)])
def test_norm_rope_write_blocks(pages, hkv, bs):
    """Block scales with other block sizes, more KV heads than a group of eight, and rows that
    begin inside blocks; a weight that is not 16-byte aligned."""
    b = Batch(LENS, NEW, hkv=hkv, bs=bs, pages=pages, scales="block", seed=bs)
    q, k, v = b.rows(hkv), b.rows(hkv), b.rows(hkv)
    w = (1 + 0.3 * torch.randn(129, generator=b.g)).bfloat16()
    rope = pgd.rope_table(max(LENS), 128)
    got = run_norm_rope(b, hkv, q, k, v, q_weight=w.cuda()[1:], k_weight=w.cuda()[:128],
                        eps=1e-6, rope=rope.cuda())
    want, size = {}, {}
    for s in range(len(LENS)):
        for row, pos in ref.rows_of(b.cu, b.lens, s):
            y, m = ref.norm_rotate(q[row], w[1:], 1e-6, rope, False, pos)
            assert torch.all((got[row].double() - y).abs() <= 2.0 ** -8 * y.abs() + F32 * m)
            want[row], size[row] = ref.norm_rotate(k[row], w[:128], 1e-6, rope, False, pos)
    check_stored(b, "k", want, size, b.dk, b.dks, F32)
    want = {r: v[r].double() for r in want}
    check_stored(b, "v", want, {r: y.abs() for r, y in want.items()}, b.dv, b.dvs, 0.0)


def test_rotation_table_too_short():
    """A sequence longer than the table is reported and left out."""
    b = Batch([20, 50, 30], [20, 10, 30], hkv=2, seed=7)
    q, k = b.rows(4), b.rows(2)
    with b_pool(b) as pool:
        before = bits(b.dk).clone()
        out = pgd.paged_qk_norm_rope_write(pool, b.to(q), b.to(k), b.to(k), *b.where(),
                                           rope=pgd.rope_table(49, 128).cuda())
        assert pgd.paged_gqa_get_error(pool) == _lib.PGD_ERR_SEQ_LEN
    assert torch.all(out[20:30].isnan()) and not out[:20].isnan().any()
    for t in range(50):
        blk, slot = ref.place(b.table, 16, 1, t)
        assert torch.equal(bits(b.dk)[blk, slot], before[blk, slot])


def test_norm_rope_in_place_and_packed():
    """q_out = q, and q_out as other columns of the packed rows q comes from."""
    b = Batch(LENS, NEW, hkv=2, seed=5)
    d, hq = 128, 4
    rope = pgd.rope_table(max(LENS), d).cuda()
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    packed = b.rows(2 * hq + 4, packed=False).cuda()
    q, k, v = packed[:, :hq], packed[:, 2 * hq:2 * hq + 2], packed[:, 2 * hq + 2:]
    with b_pool(b) as pool:
        call = lambda **kw: pgd.paged_qk_norm_rope_write(pool, q, k, v, *b.where(), q_weight=w,
                                                         k_weight=w, rope=rope, **kw)
        want = call()
        call(q_out=packed[:, hq:2 * hq])
        assert torch.equal(packed[:, hq:2 * hq], want)
        call(q_out=q)
        assert torch.equal(packed[:, :hq], want)
        with pytest.raises(pgd.PagedGQAError, match="PGD_ERR_ARG"):
            call(q_out=packed[:, 1:hq + 1])
        ok(pool)


def check_attend(b, hq, causal, window, q=None, scale=None, out=None):
    q = b.rows(hq) if q is None else q
    scale = b.d ** -0.5 if scale is None else scale
    with b_pool(b) as pool:
        got = pgd.paged_gqa_attend(pool, b.to(q), *b.where(), scale, causal=causal,
                                   window=window, out=out)
        ok(pool)
    want, size = ref.attend(q, b.k, b.v, b.k_scale, b.v_scale, b.cu, b.table, b.lens, scale,
                            causal, window)
    got = got.cpu().double()
    for row, y in want.items():
        # the weights p_t are rounded to 16 bits (at most half a step, 2^-8), scores carry
        # float32 errors (D products: below 2^-13 in p_t, in numerator and denominator),
        # and the output is rounded
        tol = 2.0 ** -8 * y.abs() + (2.0 ** -8 + 2.0 ** -12) * size[row]
        err = (got[row] - y).abs()
        assert torch.all(err <= tol), (row, float((err - tol).max()))
    return got


ATTEND_FORMS = [f for f in FORMS if f[0] != "f32"]


@pytest.mark.parametrize("bs", [8, 16, 64, 256])
@pytest.mark.parametrize("pages,scales,d", ATTEND_FORMS)
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 33)])
def test_attend(pages, scales, d, bs, causal, window):
    b = Batch(LENS, NEW, hkv=2, d=d, bs=bs, pages=pages, scales=scales, seed=bs + window, pad=2)
    out = torch.full((b.total, 6, d), 7.0, dtype=b.act, device="cuda")
    got = check_attend(b, 6, causal, window, out=out)
    assert torch.all(got[int(b.cu[-1]):] == 7)


@pytest.mark.parametrize("hkv,group", [(1, 1), (5, 1), (1, 40), (2, 7), (1, 64), (3, 130)])
def test_attend_heads(hkv, group):
    b = Batch([70, 9, 131], [5, 9, 90], hkv=hkv, seed=group)
    check_attend(b, hkv * group, True, 0)
    b = Batch([70, 9, 131], [5, 9, 90], hkv=hkv, seed=group)
    check_attend(b, hkv * group, False, 0)


@pytest.mark.parametrize("causal", [True, False])
def test_attend_long(causal):
    """Several key tiles and several query tiles a head."""
    b = Batch([1000, 517, 2], [700, 517, 1], hkv=1, bs=32, seed=9)
    check_attend(b, 4, causal, 0)


@pytest.mark.parametrize("pages", ["e4m3", "int8"])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 300)])
def test_attend_block_scales_that_vary(pages, causal, window):
    """Scales of K over a factor of 30, of V from 0 over five orders of magnitude, rising and
    falling along the sequence, in many key tiles."""
    b = Batch([1100, 700], [150, 700], hkv=2, pages=pages, scales="block", seed=3)
    for s in range(2):
        n = -(-b.lens[s] // 16)
        i = torch.arange(n, dtype=torch.float32)
        blk = b.table[s][:n].long()
        up = 10.0 ** (5 * i / n - 5) if s == 0 else 10.0 ** (-5 * i / n)
        b.v_scale[blk] *= up[:, None] * 100
        b.k_scale[blk] *= (0.2 + 6 * torch.rand(n, 1, generator=b.g)) / 6
        b.v_scale[blk[0]], b.k_scale[blk[3]] = 0.0, 0.0
    check_attend(b, 4, causal, window)


@pytest.mark.parametrize("pages,scales", [("bf16", "head"), ("e4m3", "head"), ("int8", "block")])
def test_attend_few_rows_of_long_sequences(pages, scales):
    """Sequences shared by the CTAs of a cluster: a few tokens over many key tiles."""
    b = Batch([2500, 1, 40, 1290], [3, 1, 2, 1], hkv=1, pages=pages, scales=scales, seed=5)
    for causal in (True, False):
        check_attend(b, 5, causal, 0)


def test_attend_more_queries_than_cached():
    """Cross attention has its own lengths: 300 queries over 5 tokens, 10 over none (zeros).
    Causally, queries before the first cached token see nothing."""
    for causal in (False, True):
        b = Batch([5, 0, 40], [300, 10, 64], hkv=2, seed=1)
        got = check_attend(b, 4, causal, 0)
        assert torch.all(got[300:310] == 0)


def test_attend_largest_window():
    """A window of 2^31 - 1 is none, also for queries before the first cached token."""
    b = Batch([5, 0, 40, 200], [300, 10, 64, 130], hkv=2, seed=1)
    q = b.rows(4)
    got = check_attend(b, 4, True, 2 ** 31 - 1, q=q)
    assert torch.equal(got, check_attend(b, 4, True, 0, q=q))


@pytest.mark.parametrize("pages,scales", [("bf16", "head"), ("e4m3", "block"), ("int8", "head")])
@pytest.mark.parametrize("B", [3, 12, 26])
def test_attend_shared_by_clusters_of_every_size(B, pages, scales):
    """Wide tables make clusters of 8, 4 and 2 CTAs share a piece of rows, though there are
    few key tiles: shares without a tile, blocks of 256 rows, one block and less."""
    b = Batch([700 + 16 * i for i in range(B)], [(150, 20, 200, 90)[i % 4] for i in range(B)],
              hkv=1, pages=pages, scales=scales, seed=B)
    wide = torch.full((B, 4096 - b.table.shape[1]), -1, dtype=torch.int32)
    b.table = torch.cat([b.table, wide], 1).contiguous()
    check_attend(b, 4, True, 0)
    check_attend(b, 4, False, 0)
    check_attend(b, 4, True, 100)


@pytest.mark.parametrize("pages,scales", [("bf16", "head"), ("e4m3", "head"), ("int8", "block")])
def test_attend_small_logit_scales(pages, scales):
    """A scale near the smallest float32: all weights are equal, masked tokens have none."""
    b = Batch([300, 70], [140, 70], hkv=2, pages=pages, scales=scales, seed=8)
    check_attend(b, 4, True, 40, scale=1e-37)


@pytest.mark.parametrize("pages", ["bf16", "e4m3"])
def test_attend_windows_skip_released_blocks(pages):
    """Blocks wholly before every window may be gone: table entry -1, pages poisoned."""
    b = Batch([400, 333], [30, 1], hkv=2, pages=pages, seed=2)
    for s, (x, n) in enumerate(zip(b.lens, b.new)):
        b.table[s][:max(0, x - n - 50 + 1) // 16] = -1
    check_attend(b, 8, True, 50)


def test_attend_sharp_scores():
    """Scores near +-900: one token takes all the weight, and the running maximum jumps."""
    b = Batch([600], [140], hkv=1, seed=4)
    q = (b.rows(4).float() * 9).to(torch.bfloat16)
    check_attend(b, 4, False, 0, q=q, scale=2.0)
    check_attend(b, 4, True, 0, q=q, scale=-1.0)
    check_attend(b, 4, False, 0, q=q, scale=0.0)


def test_attend_agrees_with_decode():
    """One token a sequence, and four of them: the decode entry points' answers."""
    for n in (1, 4):
        b = Batch([40, 129, 500], [n] * 3, hkv=8, seed=n)
        q = b.rows(32, packed=False)
        got = check_attend(b, 32, True, 0, q=q)
        pool = b.pool()
        dec = pgd.paged_gqa_decode_ex(pool, q.view(3, n, 32, 128).cuda(), b.table.cuda(),
                                      b.len_t.cuda(), 128 ** -0.5)
        ok(pool)
        pool.close()
        # both are within 2^-7 of the definition, relative to sums of |v| near 1
        assert (got.view(3, n, 32, 128) - dec.cpu().double()).abs().max() < 2.0 ** -5


@pytest.mark.parametrize("bad", ["len", "rows", "cu", "id"])
def test_bad_tables_are_latched(bad):
    """Impossible lengths and block ids: reported, the sequence's rows NaN, the others
    right, and nothing stored for it."""
    b = Batch([50, 60, 70], [20, 30, 40], hkv=2, seed=6)
    q, k = b.rows(4), b.rows(2)
    cu, table, lens = b.where()
    rows = slice(20, 50)
    if bad == "len":
        lens[1] = 16 * table.shape[1] + 1
    elif bad == "rows":
        lens[1] = 29
    elif bad == "cu":
        cu[3] = 500
        rows = slice(50, 90)
    else:
        table[1, 3] = b.k.shape[0]                    # positions 48 .. 59
    status = _lib.PGD_ERR_BLOCK_ID if bad == "id" else _lib.PGD_ERR_SEQ_LEN
    with b_pool(b) as pool:
        before = bits(b.dk).clone()
        dq, dk = b.to(q), b.to(k)
        kr, vr = pgd.paged_kv_read(pool, b.total, cu, table, lens)
        assert pgd.paged_gqa_get_error(pool) == status
        nan = torch.zeros(b.total, dtype=torch.bool)
        nan[slice(38, 50) if bad == "id" else rows] = True
        assert torch.equal(kr.isnan().any(2).any(1).cpu(), nan)
        out = pgd.paged_gqa_attend(pool, dq, cu, table, lens, 0.1, causal=True)
        err = pgd.paged_gqa_get_error(pool)
        if bad != "rows":                             # more queries than cached is no error there
            assert err == status
            assert torch.equal(out.isnan().any(2).any(1).cpu()[nan], nan[nan])
            assert not out[:20].isnan().any()
        qo = pgd.paged_qk_norm_rope_write(pool, dq, dk, dk, cu, table, lens)
        assert pgd.paged_gqa_get_error(pool) == status
        if bad != "id":
            assert torch.equal(qo.isnan().any(2).any(1).cpu(), nan)
        slots = torch.zeros(before.shape[:2], dtype=torch.bool)
        for s in range(3):
            for row, pos in ref.rows_of(b.cu, b.lens, s):
                if not nan[row]:
                    blk, slot = ref.place(b.table, 16, s, pos)
                    slots[blk, slot] = True
        assert torch.equal(bits(b.dk).cpu()[~slots], before.cpu()[~slots])


def test_a_step_of_a_model_layer():
    """Prompts, then single tokens, as a model runs a layer: norm, rotation and write,
    then attention of the chunk, then decode of the next token from the same pages, on one
    stream, captured into a graph and replayed; the pages read back."""
    b = Batch([45, 128, 300], [45, 60, 300], hkv=2, bs=16, pages="e4m3", scales="block", seed=8)
    hq, d = 8, 128
    rope = pgd.rope_table(512, d).cuda()
    w = (1 + 0.1 * torch.randn(d, generator=b.g)).bfloat16().cuda()
    q, k, v = b.rows(hq).cuda(), b.rows(2).cuda(), b.rows(2).cuda()
    cu, table, lens = b.where()
    pool = b.pool()
    start = [t.clone() for t in (b.dk.view(torch.uint8), b.dv.view(torch.uint8), b.dks, b.dvs)]
    dq = torch.randn((3, hq, d), generator=b.g).bfloat16().cuda()
    ws = pgd.alloc_workspace(pool, 3, hq)
    out = torch.empty((b.total, hq, d), dtype=torch.bfloat16, device="cuda")
    dec = torch.empty_like(dq)
    qo = torch.empty_like(out)
    kr = [torch.empty((b.total, 2, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    def step(s):
        pgd.paged_qk_norm_rope_write(pool, q, k, v, cu, table, lens, q_weight=w, k_weight=w,
                                     rope=rope, q_out=qo, stream=s)
        pgd.paged_gqa_attend(pool, qo, cu, table, lens, d ** -0.5, out=out, stream=s)
        pgd.paged_gqa_decode(pool, dq, table, lens, d ** -0.5, out=dec, workspace=ws, stream=s)
        pgd.paged_kv_read(pool, b.total, cu, table, lens, out=kr, stream=s)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    step(s)
    s.synchronize()
    first = [t.clone() for t in (out, dec, *kr, b.dk.view(torch.uint8), b.dks)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step(s)
    for t, x in zip((b.dk.view(torch.uint8), b.dv.view(torch.uint8), b.dks, b.dvs), start):
        t.copy_(x)
    out.zero_(), dec.zero_()
    g.replay()
    torch.cuda.synchronize()
    ok(pool)
    for x, y in zip(first, (out, dec, *kr, b.dk.view(torch.uint8), b.dks)):
        assert torch.equal(bits(x), bits(y))
    # the attention of what the pages hold now, from the definition
    now = [t.cpu() for t in (b.dk, b.dv, b.dks, b.dvs)]
    want, size = ref.attend(qo.cpu(), *now, b.cu, b.table, b.lens, d ** -0.5, True, 0)
    for row, y in want.items():
        tol = 2.0 ** -8 * y.abs() + (2.0 ** -8 + 2.0 ** -12) * size[row]
        assert torch.all((out[row].cpu().double() - y).abs() <= tol)
    last = ref.attend(dq.cpu(), *now, [0, 1, 2, 3], b.table, b.lens, d ** -0.5, False, 0)[0]
    for i, y in last.items():
        assert (dec[i].cpu().double() - y).abs().max() <= 1e-2 + 2.0 ** -8 * y.abs().max()
    pool.close()


def test_two_streams_at_once():
    """Calls on two streams, each with its own pages, give the answers they give alone."""
    bs = [Batch([300, 40], [100, 40], hkv=2, seed=s) for s in (1, 2)]
    qs = [b.to(b.rows(8)) for b in bs]
    ks = [b.to(b.rows(2)) for b in bs]
    pools = [b.pool() for b in bs]
    where = [b.where() for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    alone = []
    for p, q, k, w in zip(pools, qs, ks, where):
        pgd.paged_kv_write(p, k, k, *w)
        alone.append(pgd.paged_gqa_attend(p, q, *w, 0.09))
    torch.cuda.synchronize()
    for _ in range(20):
        outs = []
        for p, q, k, w, s in zip(pools, qs, ks, where, streams):
            pgd.paged_kv_write(p, k, k, *w, stream=s)
            outs.append(pgd.paged_gqa_attend(p, q, *w, 0.09, stream=s))
        torch.cuda.synchronize()
        for x, y in zip(outs, alone):
            assert torch.equal(x, y)
    for p in pools:
        ok(p)
        p.close()


def raw(name, *args):
    return getattr(_lib.load(), name)(*args)


def test_refusals():
    """Every status of the C entry points that needs a pool, and that a refused call
    writes nothing.  Pointers of calls that must be refused are small fake addresses."""
    A, H, AL = _lib.PGD_ERR_ARG, _lib.PGD_ERR_SHAPE, _lib.PGD_ERR_ALIGN
    b = Batch([20], [4], hkv=2, seed=1)
    pool = b.pool()
    before = bits(b.dk).clone()
    h = pool.handle
    base = dict(k=256, ks=256, v=256, vs=256, total=4, cu=256, B=1, table=256, mb=2, lens=256)
    wr = lambda **kw: (lambda a: raw("paged_kv_write", h, a["k"], a["ks"], a["v"], a["vs"],
                                     a["total"], a["cu"], a["B"], a["table"], a["mb"], a["lens"],
                                     None))({**base, **kw})
    assert wr(total=0) == _lib.PGD_OK and wr(B=0) == _lib.PGD_OK
    for kw, want in ((dict(total=-1), A), (dict(B=-1), A), (dict(mb=-1), A), (dict(mb=0), H),
                     (dict(mb=1 << 28), H), (dict(cu=None), A), (dict(table=None), A),
                     (dict(lens=None), A), (dict(cu=258), AL), (dict(k=None), A),
                     (dict(v=None), A), (dict(k=264), AL), (dict(ks=255), H), (dict(vs=0), H),
                     (dict(ks=257), AL)):
        assert wr(**kw) == want, kw
    rd = lambda k, v, total=4, B=1: raw("paged_kv_read", h, k, v, total, 256, B, 256, 2, 256, None)
    assert rd(256, 256 + 1024) == A                   # the outputs overlap
    assert rd(None, 256) == A and rd(264, 1 << 20) == AL and rd(256, 1 << 20, total=-1) == A
    nbase = dict(q=1 << 20, qs=512, o=1 << 21, os=512, hq=4, qw=None, kw=None, wd=1, eps=1e-6,
                 rope=None, rl=0, rd=0, il=0, **base)
    nr = lambda **kw: (lambda a: raw(
        "paged_qk_norm_rope_write", h, a["q"], a["qs"], a["o"], a["os"], a["hq"], a["k"], a["ks"],
        a["v"], a["vs"], a["total"], a["qw"], a["kw"], a["wd"], a["eps"], a["rope"], a["rl"],
        a["rd"], a["il"], a["cu"], a["B"], a["table"], a["mb"], a["lens"], None))({**nbase, **kw})
    for kw, want in ((dict(hq=0), A), (dict(hq=5), H), (dict(eps=-1.0), A),
                     (dict(eps=float("nan")), A), (dict(qw=256, wd=2), _lib.PGD_ERR_DTYPE),
                     (dict(il=2), A), (dict(rope=256, rl=0, rd=128), A),
                     (dict(rope=256, rl=9, rd=24), H), (dict(rope=256, rl=9, rd=144), H),
                     (dict(rope=256, rl=9, rd=0), H), (dict(rope=264, rl=9, rd=128), AL),
                     (dict(q=None), A), (dict(o=None), A), (dict(qs=500), H), (dict(os=513), AL),
                     (dict(o=(1 << 20) + 16), A), (dict(o=1 << 20, os=520), A),
                     (dict(o=256), A), (dict(v=1 << 21), A),
                     (dict(qw=257), AL), (dict(kw=258, wd=0), AL)):
        assert nr(**kw) == want, kw
    abase = dict(q=1 << 20, qs=512, total=4, hq=4, B=1, causal=1, window=0, scale=1.0, o=1 << 21,
                 mb=2)
    at = lambda **kw: (lambda a: raw(
        "paged_gqa_attend", h, a["q"], a["qs"], a["total"], a["hq"], 256, a["B"], 256, a["mb"],
        256, a["causal"], a["window"], a["scale"], a["o"], None))({**abase, **kw})
    assert at(total=0) == _lib.PGD_OK
    for kw, want in ((dict(hq=0), A), (dict(hq=3), H), (dict(causal=2), A), (dict(window=-1), A),
                     (dict(causal=0, window=4), A), (dict(scale=float("inf")), A),
                     (dict(q=None), A), (dict(o=None), A), (dict(q=(1 << 20) + 2), AL),
                     (dict(qs=511), H), (dict(qs=516), AL), (dict(o=(1 << 20) + 256), A),
                     # positions less a window would pass 31 bits
                     (dict(total=4000, mb=(1 << 27) - 64, window=9, o=1 << 26), H)):
        assert at(**kw) == want, kw
    ok(pool)
    assert torch.equal(bits(b.dk), before)
    pool.close()
    f = Batch([20], [4], hkv=2, d=64, pages="f32", seed=1)
    p32 = f.pool()
    assert raw("paged_gqa_attend", p32.handle, 1 << 20, 512, 4, 4, 256, 1, 256, 2, 256, 1, 0, 1.0,
               1 << 21, None) == _lib.PGD_ERR_UNSUPPORTED
    p32.close()
