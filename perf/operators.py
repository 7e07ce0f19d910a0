"""Cases, plain forms and 64-bit forms of the cache operators of a serving step.

Four operators work on one paged K/V cache and a ragged batch of new tokens.
Sequence b has n_b = cu_seqlens[b+1] - cu_seqlens[b] rows in the packed inputs,
and they are its last n_b cached tokens (positions L_b - n_b .. L_b - 1):

  write      K and V rows are stored in the pages, quantised as they are written
             (8-bit pages with a scale per KV head, or per block and KV head);
  read       the last n_b cached tokens come back as packed rows, dequantised;
  norm_rope  queries and keys are normed per head and rotated by their position
             in one pass; queries come back, keys and values go to the pages;
  attend     n_b query tokens attend to the sequence's pages, causally (prompts
             and chunks of prompts) or to all of them (cross attention).

Lengths and sizes belong to a case; values, page order and scales to the seed.
"""
import math

import numpy as np
import torch

own = False

CODE_MAX = {"e4m3": 448.0, "int8": 127.0}
DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn,
         "int8": torch.int8}
TINY = 2.0 ** -126     # a scale below the smallest normal number stands for an all-zero block
EPS = 1e-6


def _case(name, op, **kw):
    c = {"op": op, "B": 1, "len_lo": 1, "len_hi": 1, "new_lo": 0, "new_hi": 0, "whole": False,
         "hq": 32, "hkv": 8, "d": 128, "bs": 16, "pages": "bf16", "scales": "head",
         "causal": True, "window": 0, "norm": True, "rope_dim": 128, "interleaved": False,
         "len_seed": 1}
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one new token of each of 64 sequences into int8 pages with a scale per block: the
        # write of one decode step of one layer, where latency counts
        _case("write_step_int8", "write", B=64, len_lo=128, len_hi=4096, new_lo=1, new_hi=1,
              pages="int8", scales="block"),
        # the prompts of 32 requests into e4m3 pages with a scale per block: a prefill's write
        _case("write_prompt_e4m3", "write", B=32, len_lo=128, len_hi=4096, whole=True,
              pages="e4m3", scales="block"),
        # chunks of odd lengths of long prompts, 40 KV heads, one scale per head
        _case("write_chunk_int8_head", "write", B=7, len_lo=700, len_hi=4096, new_lo=1,
              new_hi=700, hkv=40, pages="int8", scales="head"),
        # a few short shared prefixes of a small model read back from small pages
        _case("read_prefix_bf16", "read", B=5, len_lo=1, len_hi=300, whole=True, hkv=2, d=64,
              bs=8),
        # every sequence of a serving batch dequantised, as to move it or to rebuild its pages
        _case("read_batch_e4m3", "read", B=64, len_lo=128, len_hi=4096, whole=True,
              pages="e4m3", scales="block"),
        # the projections of one decode step, 64 sequences
        _case("norm_rope_step", "norm_rope", B=64, len_lo=128, len_hi=4096, new_lo=1, new_hi=1),
        # the projections of 32 prompts
        _case("norm_rope_prompt", "norm_rope", B=32, len_lo=128, len_hi=4096, whole=True),
        # chunks of long prompts, 64 query heads, into e4m3 pages with a scale per block
        _case("norm_rope_chunk_e4m3", "norm_rope", B=3, len_lo=32768, len_hi=65536, new_lo=4000,
              new_hi=8192, hq=64, bs=32, pages="e4m3", scales="block"),
        # a few tokens of eight sequences attend to encoder states: the latency of cross attention
        _case("cross_few", "attend", B=8, len_lo=128, len_hi=4096, new_lo=2, new_hi=8,
              causal=False),
        # whole prompts attend to themselves: a prefill's attention
        _case("prompt", "attend", B=4, len_lo=128, len_hi=4096, whole=True),
        # one chunk of a long prompt attends to what is cached of it
        _case("chunk_long", "attend", B=1, len_lo=32768, len_hi=32768, new_lo=2048, new_hi=2048,
              hq=64, bs=32),
        # chunks of prompts over e4m3 pages with a scale per block
        _case("chunk_e4m3", "attend", B=2, len_lo=4096, len_hi=16384, new_lo=700, new_hi=1500,
              pages="e4m3", scales="block"),
    ]


def _log(rng, lo, hi):
    """An integer spread evenly over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    while True:
        op = rng.choice(("write", "read", "norm_rope", "attend"))
        d = rng.choice((64, 128, 128))
        pages = rng.choice(("bf16", "e4m3", "int8") if d == 128 else ("bf16",))
        if op != "attend" and rng.random() < 0.15:
            pages = "f32"
        if op == "norm_rope" and pages == "int8":
            pages = "e4m3"       # whole numbers have to be equal, and sums of squares are not
        hkv = rng.choice((1, 2, 3, 4, 5, 8, 8, 10, 16, 40))
        group = rng.choice((1, 2, 3, 4, 4, 5, 7, 8, 16))
        B = _log(rng, 1, 64 if op != "attend" else 16)
        hi = _log(rng, 8, 8192)
        lo = rng.randint(1, hi)
        whole = rng.random() < 0.4
        new_hi = 1 if rng.random() < 0.3 else _log(rng, 1, hi)
        c = _case(None, op, B=B, len_lo=lo, len_hi=hi, whole=whole,
                  new_lo=0 if whole else rng.randint(0, new_hi), new_hi=0 if whole else new_hi,
                  hq=hkv * group, hkv=hkv, d=d, bs=rng.choice((8, 16, 16, 32, 64, 128, 256)),
                  pages=pages, scales=rng.choice(("head", "block")),
                  causal=rng.random() < 0.6, norm=rng.random() < 0.7,
                  rope_dim=rng.choice((d, d, d // 2)), interleaved=rng.random() < 0.3,
                  len_seed=rng.randint(1, 1 << 30))
        if op == "attend" and c["causal"] and rng.random() < 0.25:
            c["window"] = _log(rng, 1, hi)
        if c["hq"] > 128 or not sum(_lengths(c)[1]):
            continue
        w = work(c)
        lens, new = _lengths(c)
        dense = B * c["hq"] * max(new) * max(lens) if op == "attend" else 0
        rows = B * max(new) * (c["hq"] + 2 * hkv) * d
        if w["bytes"] < 1.2e9 and w["flops"] < 1.5e12 and dense < 3e9 and rows < 2e9:
            return c


def _lengths(c):
    """(cached tokens, new tokens) of each sequence, as lists."""
    r = np.random.default_rng(c["len_seed"])
    lens = r.integers(c["len_lo"], c["len_hi"] + 1, size=c["B"])
    new = lens.copy() if c["whole"] else np.minimum(
        lens, r.integers(c["new_lo"], c["new_hi"] + 1, size=c["B"]))
    return [int(x) for x in lens], [int(x) for x in new]


def work(c):
    lens, new = _lengths(c)
    T, row = sum(new), c["hkv"] * c["d"]
    elt = {"f32": 4, "bf16": 2, "e4m3": 1, "int8": 1}[c["pages"]]
    act = 4 if c["pages"] == "f32" else 2
    blocks = sum(-(-x // c["bs"]) - (x - n) // c["bs"] for x, n in zip(lens, new) if n)
    scales = 0
    if c["pages"] in CODE_MAX:
        scales = 8 * c["hkv"] * (blocks if c["scales"] == "block" else 1)
    tables = 4 * (2 * c["B"] + 1 + blocks)
    if c["op"] in ("write", "read"):
        return {"bytes": 2 * T * row * (act + elt) + scales + tables, "flops": 2 * T * row}
    if c["op"] == "norm_rope":
        q = T * c["hq"] * c["d"]
        table = 4 * c["rope_dim"] * T
        return {"bytes": 2 * q * act + 2 * T * row * (act + elt) + scales + tables + table,
                "flops": 10 * (q + T * row)}
    pairs, kv = 0, 0
    for x, n in zip(lens, new):
        if not n:
            continue
        if not c["causal"]:
            pairs, kv = pairs + n * x, kv + x
        else:
            w = c["window"] or x
            p = np.arange(x - n, x)
            pairs += int(np.minimum(p + 1, w).sum())
            kv += x - max(0, x - n - w + 1)
    if c["pages"] in CODE_MAX:
        scales = 8 * c["hkv"] * (-(-kv // c["bs"]) if c["scales"] == "block" else 1)
    return {"bytes": 2 * T * c["hq"] * c["d"] * 2 + 2 * kv * row * elt + scales
            + 4 * (2 * c["B"] + 1 + -(-kv // c["bs"])),
            "flops": 4 * pairs * c["hq"] * c["d"]}


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    lens, new = _lengths(c)
    nbs = [-(-x // c["bs"]) for x in lens]
    used, mb = sum(nbs), max(max(nbs), 1)
    nb = used + used // 10 + 2            # the last block stays out of every table
    perm = torch.randperm(nb - 1, generator=g, device=dev)[:used].to(torch.int32)
    table = torch.full((c["B"], mb), -1, dtype=torch.int32, device=dev)
    valid = (torch.arange(mb, device=dev)[None]
             < torch.tensor(nbs, device=dev)[:, None])
    table[valid] = perm
    T = sum(new)
    act = torch.float32 if c["pages"] == "f32" else torch.bfloat16
    s = {"case": c, "T": T, "max_len": max(lens), "max_new": max(new),
         "table": table,
         "lens": torch.tensor(lens, dtype=torch.int32, device=dev),
         "cu": torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device=dev)}

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    shape = (nb, c["bs"], c["hkv"], c["d"])
    if c["pages"] in CODE_MAX:
        top = CODE_MAX[c["pages"]]
        for x in ("k", "v"):
            codes = (randn(*shape) * (top / 4.5)).clamp_(-top, top)
            s[x] = (codes.round_() if c["pages"] == "int8" else codes).to(DTYPE[c["pages"]])
            by = (nb, c["hkv"]) if c["scales"] == "block" else (c["hkv"],)
            s[x + "_scale"] = (0.7 + 0.6 * torch.rand(by, generator=g, device=dev)) * (4.5 / top)
    else:
        s["k"], s["v"] = randn(*shape).to(act), randn(*shape).to(act)
        s["k_scale"] = s["v_scale"] = None
    if c["op"] in ("write", "norm_rope"):
        # queries, keys and values as one projection leaves them: views of a packed row
        nq = c["hq"] if c["op"] == "norm_rope" else 0
        rows = randn(T, nq + 2 * c["hkv"], c["d"])
        rows *= 0.5 + torch.rand((1, nq + 2 * c["hkv"], 1), generator=g, device=dev)
        rows = rows.to(act)
        s["q_new"] = rows[:, :nq]
        s["k_new"], s["v_new"] = rows[:, nq:nq + c["hkv"]], rows[:, nq + c["hkv"]:]
    if c["op"] == "norm_rope":
        half = c["rope_dim"] // 2
        freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
        ang = torch.arange(max(lens), dtype=torch.float64, device=dev)[:, None] * freq
        s["rope"] = torch.stack((ang.cos(), ang.sin()), 1).float()    # [max_len, 2, half]
        s["q_weight"] = (1 + 0.2 * randn(c["d"])).to(act) if c["norm"] else None
        s["k_weight"] = (1 + 0.2 * randn(c["d"])).to(act) if c["norm"] else None
    if c["op"] == "attend":
        s["q"] = randn(T, c["hq"], c["d"]).to(act)
        s["scale"] = 1.0 / math.sqrt(c["d"])
    if own:
        import paged_gqa_decode_04_gb300 as pgd

        s["pgd"] = pgd
        s["pool"] = pgd.PagedKVPool(s["k"], s["v"], s["k_scale"], s["v_scale"])
        act_empty = dict(dtype=act, device=dev)
        if c["op"] == "read":
            s["out"] = [torch.empty((T, c["hkv"], c["d"]), **act_empty) for _ in range(2)]
        elif c["op"] != "write":
            s["out"] = torch.empty((T, c["hq"], c["d"]), **act_empty)
    return s


def _pages(s):
    """The cache after a write: pages, and scales where the pages are 8-bit."""
    return [s[x] for x in ("k", "v", "k_scale", "v_scale") if s[x] is not None]


def _run_own(s):
    c, pgd = s["case"], s["pgd"]
    where = (s["cu"], s["table"], s["lens"])
    if c["op"] == "write":
        pgd.paged_kv_write(s["pool"], s["k_new"], s["v_new"], *where)
        return _pages(s)
    if c["op"] == "read":
        return list(pgd.paged_kv_read(s["pool"], s["T"], *where, out=s["out"]))
    if c["op"] == "norm_rope":
        q = pgd.paged_qk_norm_rope_write(
            s["pool"], s["q_new"], s["k_new"], s["v_new"], *where, q_weight=s["q_weight"],
            k_weight=s["k_weight"], eps=EPS, rope=s["rope"], interleaved=c["interleaved"],
            q_out=s["out"])
        return [q] + _pages(s)
    return pgd.paged_gqa_attend(s["pool"], s["q"], *where, s["scale"], causal=c["causal"],
                                window=c["window"], out=s["out"])


# ------------------------------------------------------------------ plain forms

def _places(s):
    """Sequence and position of each packed row, its physical block and slot."""
    c = s["case"]
    cu, lens = s["cu"].long(), s["lens"].long()
    n = cu[1:] - cu[:-1]
    b = torch.repeat_interleave(torch.arange(c["B"], device=cu.device), n, output_size=s["T"])
    pos = lens[b] - n[b] + torch.arange(s["T"], device=cu.device) - cu[b]
    return b, pos, s["table"].long()[b, pos // c["bs"]], pos % c["bs"]


def _codes(x, pages):
    """Codes of values already divided by their scale."""
    top = CODE_MAX[pages]
    x = x.clamp(-top, top)
    return (x.round() if pages == "int8" else x).to(DTYPE[pages])


def _bits(t):
    return t.view(torch.uint8) if t.element_size() == 1 else t


def _inverse(scale):
    return torch.where(scale > 0, 1.0 / scale, torch.zeros_like(scale))


def _store(s, x, rows, blk, slot):
    """Store float32 rows [T, Hkv, D] in pool `x`, quantised where it is 8-bit."""
    c, pool, sc = s["case"], s[x], s[x + "_scale"]
    if sc is None:
        pool[blk, slot] = rows.to(pool.dtype)
        return
    if c["scales"] == "head":
        _bits(pool)[blk, slot] = _bits(_codes(rows * _inverse(sc)[:, None], c["pages"]))
        return
    # a block's scale covers what it holds: the rows cached in it before (a sequence's first
    # block of this call, where the call begins inside it) and the new ones
    cu, lens = s["cu"].long(), s["lens"].long()
    n = cu[1:] - cu[:-1]
    start = lens - n
    kept = torch.where(n > 0, start % c["bs"], 0)
    trash = pool.shape[0] - 1
    at = (start // c["bs"]).clamp(max=s["table"].shape[1] - 1)
    first = torch.where(kept > 0, s["table"].long().gather(1, at[:, None])[:, 0], trash)
    old = torch.where((kept > 0)[:, None], sc[first], 0.0)            # [B, Hkv]
    new = torch.zeros_like(sc)
    idx = blk[:, None].expand(-1, c["hkv"])
    new.scatter_reduce_(0, idx, rows.abs().amax(-1), "amax")
    new = new / CODE_MAX[c["pages"]]
    new = torch.where(new >= TINY, new, 0.0)
    new.scatter_reduce_(0, first[:, None].expand_as(old), old, "amax")
    touched = torch.zeros(pool.shape[0], dtype=torch.bool, device=pool.device)
    touched[blk] = True
    # rows cached before, at the scale that the block has now
    ratio = torch.where(new[first] > old, old * _inverse(new[first]), 1.0)
    was = pool[first].float() * ratio[:, None, :, None]
    keep = (torch.arange(c["bs"], device=pool.device)[None] < kept[:, None])[:, :, None, None]
    _bits(pool)[first] = torch.where(keep, _bits(_codes(was, c["pages"])), _bits(pool)[first])
    sc.copy_(torch.where(touched[:, None], new, sc))
    _bits(pool)[blk, slot] = _bits(_codes(rows * _inverse(new)[blk][:, :, None], c["pages"]))


def _load(s, x, blk, slot):
    """float32 values of pool `x` at the given blocks and slots."""
    pool, sc = s[x], s[x + "_scale"]
    rows = (_bits(pool)[blk, slot]).view(pool.dtype).float()
    if sc is None:
        return rows
    return rows * (sc[:, None] if s["case"]["scales"] == "head" else sc[blk][..., None])


def _normed_rotated(x, weight, cos, sin, interleaved):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    half = cos.shape[-1]
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = r[..., :half], r[..., half:]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((r, rest), -1)


def _attend(s):
    """Dense scores of every sequence, padded to the longest, and a masked softmax."""
    c = s["case"]
    cu, lens, table = s["cu"].long(), s["lens"].long(), s["table"].long()
    n = cu[1:] - cu[:-1]
    dev = cu.device
    t = torch.arange(s["max_len"], device=dev)
    blk = table[:, t // c["bs"]].clamp(min=0)                         # [B, Lmax]
    there = (t[None] < lens[:, None])[:, :, None, None]
    k = torch.where(there, _load(s, "k", blk, (t % c["bs"])[None]), 0.0)
    v = torch.where(there, _load(s, "v", blk, (t % c["bs"])[None]), 0.0)
    i = torch.arange(s["max_new"], device=dev)
    rows = (cu[:-1, None] + i[None]).clamp(max=s["T"] - 1)            # [B, nmax]
    group = c["hq"] // c["hkv"]
    q = s["q"][rows].float().view(c["B"], s["max_new"], c["hkv"], group, c["d"])
    q = q.permute(0, 2, 3, 1, 4).reshape(c["B"], c["hkv"], group * s["max_new"], c["d"])
    p = (q * s["scale"]) @ k.permute(0, 2, 3, 1)                      # [B, Hkv, G nmax, Lmax]
    p = p.view(c["B"], c["hkv"], group, s["max_new"], s["max_len"])
    at = lens[:, None] - n[:, None] + i[None]                         # query positions [B, nmax]
    see = (t[None, None] < lens[:, None, None]).expand(-1, s["max_new"], -1)
    if c["causal"]:
        see = see & (t[None, None] <= at[:, :, None])
        if c["window"]:
            see = see & (t[None, None] > at[:, :, None] - c["window"])
    p.masked_fill_(~see[:, None, None], float("-inf"))
    top = p.amax(-1, keepdim=True)
    p.sub_(torch.where(torch.isfinite(top), top, 0.0)).exp_()
    total = p.sum(-1)
    o = p.view(c["B"], c["hkv"], group * s["max_new"], s["max_len"]) @ v.permute(0, 2, 1, 3)
    o = o.view(c["B"], c["hkv"], group, s["max_new"], c["d"])
    o = o / torch.where(total > 0, total, 1.0)[..., None]
    o = o.permute(0, 3, 1, 2, 4).reshape(c["B"], s["max_new"], c["hq"], c["d"])
    b = torch.repeat_interleave(torch.arange(c["B"], device=dev), n, output_size=s["T"])
    return o[b, torch.arange(s["T"], device=dev) - cu[b]].to(s["q"].dtype)


def run(state):
    s = state
    if own:
        return _run_own(s)
    c = s["case"]
    if c["op"] == "attend":
        return _attend(s)
    b, pos, blk, slot = _places(s)
    if c["op"] == "read":
        act = torch.float32 if c["pages"] == "f32" else torch.bfloat16
        return [_load(s, x, blk, slot).to(act) for x in ("k", "v")]
    if c["op"] == "write":
        _store(s, "k", s["k_new"].float(), blk, slot)
        _store(s, "v", s["v_new"].float(), blk, slot)
        return _pages(s)
    cos, sin = s["rope"][pos].unbind(1)
    q = _normed_rotated(s["q_new"], s["q_weight"], cos, sin, c["interleaved"]).to(s["q_new"].dtype)
    _store(s, "k", _normed_rotated(s["k_new"], s["k_weight"], cos, sin, c["interleaved"]),
           blk, slot)
    _store(s, "v", s["v_new"].float(), blk, slot)
    return [q] + _pages(s)


# ------------------------------------------------------- 64-bit forms, row by row

def _nearest_code(x, pages):
    """The nearest code's value, ties to even, saturated: by the spacing of the code at x."""
    if pages == "int8":
        return torch.round(x).clamp(-127, 127)
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_store(s, pool, scale, rows, lens, new, table):
    """pool, scale (float64) after the rows are stored, sequence by sequence."""
    c = s["case"]
    bs, at = c["bs"], 0
    for b, (x, n) in enumerate(zip(lens, new)):
        for i in range((x - n) // bs, -(-x // bs) if n else 0):
            lo, hi = max(x - n, i * bs), min(x, (i + 1) * bs)
            blk, first = table[b][i], lo - i * bs
            part = rows[at:at + hi - lo]
            at += hi - lo
            if scale is None:
                pool[blk, first:first + hi - lo] = part
                continue
            if c["scales"] == "block":
                top = part.abs().amax((0, 2)) / CODE_MAX[c["pages"]]
                if first:
                    was = scale[blk].clone()
                    top = torch.maximum(top, was)
                    pool[blk, :first] = _nearest_code(
                        pool[blk, :first] * (was / top.clamp(min=TINY))[:, None], c["pages"])
                scale[blk] = top
            by = scale[blk] if c["scales"] == "block" else scale
            pool[blk, first:first + hi - lo] = _nearest_code(
                part / by.clamp(min=TINY)[:, None], c["pages"])


def _exact_rotated(x, weight, pos, c):
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["d"] + EPS) * weight.double()
    half = c["rope_dim"] // 2
    j = torch.arange(half, device=x.device)
    one, two = (2 * j, 2 * j + 1) if c["interleaved"] else (j, j + half)
    angle = pos.double()[:, None] * torch.exp(-math.log(10000.0) * j.double() / half)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    z = torch.complex(x[..., one], x[..., two]) * turn
    y = x.clone()
    y[..., one], y[..., two] = z.real, z.imag
    return y


def exact(case, seed):
    c = dict(case)
    lens, new = _lengths(c)
    if c["op"] in ("write", "norm_rope") and \
            sum(-(-x // c["bs"]) - (x - n) // c["bs"] for x, n in zip(lens, new) if n) > 20000:
        return None
    s = prepare(c, seed)
    dev = s["cu"].device
    table = s["table"].tolist()

    def cached(x, b, lo, hi):
        """Values of tokens lo .. hi-1 of sequence b, [hi - lo, Hkv, D]."""
        t = torch.arange(lo, hi, device=dev)
        blk = s["table"][b].long()[t // c["bs"]]
        val = s[x].view(torch.uint8 if s[x].element_size() == 1 else s[x].dtype)
        val = val[blk, t % c["bs"]].view(s[x].dtype).double()
        if s[x + "_scale"] is not None:
            sc = s[x + "_scale"].double()
            val = val * (sc[None, :, None] if c["scales"] == "head" else sc[blk][:, :, None])
        return val

    if c["op"] == "read":
        return [torch.cat([cached(x, b, y - n, y) for b, (y, n) in enumerate(zip(lens, new))])
                for x in ("k", "v")]
    if c["op"] == "attend":
        out = torch.zeros(s["T"], c["hq"], c["d"], dtype=torch.float64, device=dev)
        at, group = 0, c["hq"] // c["hkv"]
        for b, (x, n) in enumerate(zip(lens, new)):
            if not n:
                continue
            k, v = cached("k", b, 0, x), cached("v", b, 0, x)
            p = torch.arange(x - n, x, device=dev)
            t = torch.arange(x, device=dev)
            hide = t[None] > p[:, None] if c["causal"] else torch.zeros(n, x, dtype=torch.bool,
                                                                        device=dev)
            if c["causal"] and c["window"]:
                hide |= t[None] <= p[:, None] - c["window"]
            for h in range(c["hq"]):
                z = s["q"][at:at + n, h].double() @ k[:, h // group].T * s["scale"]
                w = torch.softmax(z.masked_fill(hide, float("-inf")), -1)
                out[at:at + n, h] = w @ v[:, h // group]
            at += n
        return out
    whole = c["pages"] == "int8"
    k, v = s["k"].double(), s["v"].double()
    ks, vs = (None if s[x] is None else s[x].double() for x in ("k_scale", "v_scale"))
    pos = torch.tensor([p for x, n in zip(lens, new) for p in range(x - n, x)], device=dev)
    kn = s["k_new"].double()
    if c["op"] == "norm_rope":
        kn = _exact_rotated(s["k_new"], s["k_weight"], pos, c)
    _exact_store(s, k, ks, kn, lens, new, table)
    _exact_store(s, v, vs, s["v_new"].double(), lens, new, table)
    pages = [None if whole else k, None if whole else v] + ([] if ks is None else [ks, vs])
    if c["op"] == "norm_rope":
        return [_exact_rotated(s["q_new"], s["q_weight"], pos, c)] + pages
    return pages
