"""Cases, plain forms and 64-bit forms of attention with shaped scores and of decode with
shared prefixes.

Three operators read one paged K/V cache.  A query at position p scores token t as

  s = scale <q, k_t>;  s <- softcap tanh(s / softcap);  s <- s - slope_h |p - t|

(each of the last two steps where it is asked for), and attends to what causality, a window
and its own visible range leave of the L cached tokens:

  attend  ragged queries over the pages: prompts, chunks of prompts, packed documents, prefix
          masks.  Sequence b owns rows cu_seqlens[b] .. cu_seqlens[b+1] - 1, query i of n at
          p = L - n + i;
  decode  the last one to a few cached tokens of every sequence are the queries;
  shared  the same for groups of sequences whose first shared_lens[g] tokens are the same
          ones: forks of one prompt, whose tables name the same blocks.

Lengths and sizes belong to a case; values, page order and scales to the seed.
"""
import math

import numpy as np
import torch

own = False

CODE_MAX = {"e4m3": 448.0, "int8": 127.0}
DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn,
         "int8": torch.int8}


def _case(name, op, **kw):
    c = {"op": op, "B": 1, "len_lo": 1, "len_hi": 1, "new_lo": 0, "new_hi": 0, "whole": False,
         "hq": 32, "hkv": 8, "d": 128, "bs": 16, "pages": "bf16", "scales": "head",
         "causal": True, "window": 0, "cap": 0.0, "bias": False, "mask": "none", "doc_lo": 1,
         "doc_hi": 1, "blank": 0, "q_len": 1, "groups": 1, "pre_lo": 0, "pre_hi": 0,
         "len_seed": 1}
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # a few drafted tokens of eight sequences, capped: where the latency of a call counts
        _case("attend_few_cap", "attend", B=8, len_lo=128, len_hi=4096, new_lo=2, new_hi=8,
              cap=50.0),
        # a prefill's whole prompts, capped
        _case("attend_prompt_cap", "attend", B=4, len_lo=128, len_hi=4096, whole=True, cap=50.0),
        # one chunk of a long prompt with a bias that grows with distance
        _case("attend_chunk_bias", "attend", B=1, len_lo=8192, len_hi=8192, new_lo=2048,
              new_hi=2048, hq=64, bs=32, bias=True),
        # documents packed into one sequence, each attending to itself
        _case("attend_documents", "attend", B=1, len_lo=16384, len_hi=16384, whole=True,
              mask="docs", doc_lo=100, doc_hi=2000),
        # prompts whose first part is seen by all of it, capped, over e4m3 pages with block scales
        _case("attend_prefix_e4m3_cap", "attend", B=3, len_lo=700, len_hi=4096, whole=True,
              causal=False, mask="prefix", cap=30.0, pages="e4m3", scales="block"),
        # one decode step of 64 sequences, capped
        _case("decode_step_cap", "decode", B=64, len_lo=128, len_hi=4096, cap=50.0),
        # a small model's step with a bias: latency
        _case("decode_small_bias", "decode", B=4, len_lo=1, len_hi=300, hq=8, hkv=2, d=64,
              bias=True),
        # long contexts over e4m3 pages, capped and with a bias
        _case("decode_long_e4m3", "decode", B=8, len_lo=32768, len_hi=65536, hq=64, bs=32,
              bias=True, cap=50.0, pages="e4m3"),
        # 64 requests behind one long system prompt
        _case("shared_prompt", "shared", B=64, pre_lo=16384, pre_hi=16384, len_lo=128,
              len_hi=1024),
        # four prompts with eight samples each, soon after they were forked: latency
        _case("shared_samples", "shared", B=32, groups=4, pre_lo=300, pre_hi=2000, len_lo=1,
              len_hi=64),
        # three drafted tokens of 16 requests behind one prompt, 20 query heads, one KV head
        _case("shared_draft_mqa", "shared", B=16, q_len=3, hq=20, hkv=1, pre_lo=8192,
              pre_hi=8192, len_lo=64, len_hi=512),
        # 128 requests of a large model behind two long prompts over e4m3 pages, capped
        _case("shared_long_e4m3", "shared", B=128, groups=2, hq=64, bs=32, pre_lo=32768,
              pre_hi=32768, len_lo=128, len_hi=2048, pages="e4m3", cap=50.0),
    ]


def _log(rng, lo, hi):
    """An integer spread evenly over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    while True:
        op = rng.choice(("attend", "decode", "shared"))
        d = rng.choice((64, 128, 128))
        pages = rng.choice(("bf16", "bf16", "e4m3", "int8") if d == 128 else ("bf16",))
        hkv = rng.choice((1, 2, 3, 4, 5, 8, 8, 10, 16))
        group = rng.choice((1, 2, 3, 4, 4, 5, 7, 8, 16))
        hi = _log(rng, 8, 8192)
        c = _case(None, op, len_lo=rng.randint(1, hi), len_hi=hi, hq=hkv * group, hkv=hkv, d=d,
                  bs=rng.choice((8, 16, 16, 32, 64, 128, 256)), pages=pages,
                  scales=rng.choice(("head", "block")), cap=rng.choice((0.0, 20.0, 30.0, 50.0)),
                  bias=rng.random() < 0.4, len_seed=rng.randint(1, 1 << 30))
        if op == "attend":
            whole = rng.random() < 0.5
            new_hi = _log(rng, 1, hi)
            c.update(B=_log(rng, 1, 16), whole=whole, new_lo=0 if whole else rng.randint(0, new_hi),
                     new_hi=0 if whole else new_hi, mask=rng.choice(("none", "docs", "prefix")),
                     causal=rng.random() < 0.6, blank=rng.choice((0, 0, 17)))
            c["doc_hi"] = _log(rng, 1, hi)
            c["doc_lo"] = rng.randint(1, c["doc_hi"])
            if c["mask"] == "prefix":
                c["causal"] = False
            if c["causal"] and rng.random() < 0.25:
                c["window"] = _log(rng, 1, hi)
        else:
            c["q_len"] = rng.choice((1, 1, 1, 2, 3)) if group <= 16 else 1
            c["B"] = _log(rng, 1, 64)
        if op == "shared":
            c["groups"] = _log(rng, 1, min(8, c["B"]))
            c["pre_hi"] = _log(rng, 8, 32768)
            c["pre_lo"] = rng.randint(0, c["pre_hi"])
            c["len_lo"] = max(c["len_lo"], c["q_len"])
            c["len_hi"] = max(c["len_hi"], c["len_lo"])
        elif op == "decode":
            if pages == "bf16" and rng.random() < 0.1:
                c.update(pages="f32", q_len=1)
            elif rng.random() < 0.2:
                c["window"] = _log(rng, 1, hi)
        if not (c["cap"] or c["bias"] or c["mask"] != "none" or op == "shared"):
            continue
        if c["hq"] > 128 or not sum(_lengths(c)[1]):
            continue
        w = work(c)
        lens, new = _lengths(c)
        dense = c["B"] * c["hq"] * max(new) * max(lens)
        if w["bytes"] < 8e8 and w["flops"] < 1.5e11 and dense < 1e9 and \
                c["B"] * max(lens) * hkv * d < 1e9:
            return c


def _lengths(c):
    """(cached tokens, query tokens) of each sequence, as lists.  shared: cached tokens are the
    group's prefix and the sequence's own."""
    r = np.random.default_rng(c["len_seed"])
    lens = r.integers(c["len_lo"], c["len_hi"] + 1, size=c["B"])
    if c["op"] == "attend":
        new = lens.copy() if c["whole"] else np.minimum(
            lens, r.integers(c["new_lo"], c["new_hi"] + 1, size=c["B"]))
    else:
        new = np.full(c["B"], c["q_len"])
    if c["op"] == "shared":
        cu, pre = _groups(c)
        lens = lens + np.repeat(pre, np.diff(cu))
    return [int(x) for x in lens], [int(x) for x in new]


def _groups(c):
    """First sequence of each group (and B), and the prefix's tokens of each."""
    r = np.random.default_rng(c["len_seed"] + 1)
    cu = [c["B"] * g // c["groups"] for g in range(c["groups"] + 1)]
    pre = r.integers(c["pre_lo"], c["pre_hi"] + 1, size=c["groups"])
    return cu, [int(x) for x in pre]


def _visible(c, lens, new):
    """[total, 2] tokens [first, end) that each packed row of `attend` may see by its mask, or
    None."""
    if c["mask"] == "none" and not c["blank"]:
        return None
    r = np.random.default_rng(c["len_seed"] + 2)
    out = []
    for x, n in zip(lens, new):
        p = np.arange(x - n, x)
        rows = np.stack((np.zeros(n), np.full(n, x)), 1)
        if c["mask"] == "docs":
            ends = np.cumsum(r.integers(c["doc_lo"], c["doc_hi"] + 1, size=x // c["doc_lo"] + 1))
            i = np.searchsorted(ends, p, side="right")
            rows = np.stack((np.where(i > 0, ends[i - 1], 0), np.minimum(ends[i], x)), 1)
        elif c["mask"] == "prefix":
            rows[:, 1] = np.maximum(p + 1, r.integers(0, x + 1))
        if c["blank"]:
            rows[p % c["blank"] == 0, 1] = 0         # padding tokens, which see nothing
        out.append(rows)
    return np.concatenate(out).astype(np.int32)


def _seen(c, lens, new):
    """[total, 2] tokens [lo, hi) that each row sees."""
    v, out, at = _visible(c, lens, new), [], 0
    for x, n in zip(lens, new):
        p = np.arange(x - n, x)
        lo, hi = np.zeros(n, np.int64), np.full(n, x)
        if c["causal"]:
            hi = p + 1
            if c["window"]:
                lo = np.maximum(0, p - c["window"] + 1)
        if v is not None:
            lo, hi = np.maximum(lo, v[at:at + n, 0]), np.minimum(hi, v[at:at + n, 1])
        out.append(np.stack((lo, np.maximum(hi, lo)), 1))
        at += n
    return np.concatenate(out)


def work(c):
    lens, new = _lengths(c)
    elt = {"f32": 4, "bf16": 2, "e4m3": 1, "int8": 1}[c["pages"]]
    act = 4 if c["pages"] == "f32" else 2
    seen, at, kv = _seen(c, lens, new), 0, 0
    pairs = int((seen[:, 1] - seen[:, 0]).sum())
    for x, n in zip(lens, new):
        s = seen[at:at + n]
        s = s[s[:, 1] > s[:, 0]]
        kv += int(s[:, 1].max() - s[:, 0].min()) if len(s) else 0
        at += n
    if c["op"] == "shared":
        cu, pre = _groups(c)
        kv -= sum(p * (b - a - 1) for a, b, p in zip(cu, cu[1:], pre))
    blocks = -(-kv // c["bs"])
    scales = 0
    if c["pages"] in CODE_MAX:
        scales = 8 * c["hkv"] * (blocks if c["scales"] == "block" else 1)
    masks = 8 * sum(new) if c["mask"] != "none" or c["blank"] else 0
    return {"bytes": 2 * sum(new) * c["hq"] * c["d"] * act + 2 * kv * c["hkv"] * c["d"] * elt
            + scales + masks + 4 * (2 * c["B"] + 1 + blocks),
            "flops": 4 * pairs * c["hq"] * c["d"]}


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    lens, new = _lengths(c)
    bs = c["bs"]
    nbs = [-(-x // bs) for x in lens]
    table = np.full((c["B"], max(max(nbs), 1)), -1, dtype=np.int32)
    used, copies = 0, []
    cu, pre = _groups(c) if c["op"] == "shared" else (list(range(c["B"] + 1)), [0] * c["B"])
    for first, end, p in zip(cu, cu[1:], pre):
        for b in range(first, end):
            kept = p // bs if b > first else 0        # blocks of the group's first sequence
            table[b, :kept] = table[first, :kept]
            table[b, kept:nbs[b]] = np.arange(used, used + nbs[b] - kept)
            used += nbs[b] - kept
            if b > first and p % bs:                  # the prefix's last tokens, copied
                copies.append((table[first, kept], table[b, kept]))
    nb = used + used // 10 + 2
    perm = torch.randperm(nb, generator=g, device=dev).to(torch.int32)
    table = torch.from_numpy(table).to(dev)
    table = torch.where(table >= 0, perm[table.clamp(min=0).long()], table)
    act = torch.float32 if c["pages"] == "f32" else torch.bfloat16
    s = {"case": c, "T": sum(new), "max_len": max(lens), "max_new": max(new), "table": table,
         "lens": torch.tensor(lens, dtype=torch.int32, device=dev),
         "cu": torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device=dev)}

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    shape = (nb, bs, c["hkv"], c["d"])
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
    if copies:
        src, dst = perm[torch.tensor(copies, device=dev).long().T].long()
        for x in ("k", "v"):
            _bits(s[x])[dst] = _bits(s[x])[src]
            if c["scales"] == "block" and s[x + "_scale"] is not None:
                s[x + "_scale"][dst] = s[x + "_scale"][src]
    # scores that single tokens out, and that reach into the range where a cap bends them
    q = (randn(s["T"], c["hq"], c["d"]) * (4.0 if c["cap"] else 2.0)).to(act)
    s["q"] = q if c["op"] == "attend" else q.view(c["B"], c["q_len"], c["hq"], c["d"])
    s["scale"] = 1.0 / math.sqrt(c["d"])
    s["slopes"] = None
    if c["bias"]:
        h = torch.arange(1, c["hq"] + 1, dtype=torch.float64, device=dev)
        s["slopes"] = torch.exp2(-8.0 * h / c["hq"]).float()
    v = _visible(c, lens, new) if c["op"] == "attend" else None
    s["visible"] = None if v is None else torch.from_numpy(v).to(dev)
    s["groups"] = list(zip(cu, cu[1:], pre))
    s["cu_groups"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    s["shared_lens"] = torch.tensor(pre, dtype=torch.int32, device=dev)
    if own:
        import paged_gqa_decode_04_gb300 as pgd

        s["pgd"] = pgd
        s["pool"] = pgd.PagedKVPool(s["k"], s["v"], s["k_scale"], s["v_scale"])
        s["out"] = torch.empty_like(s["q"])
        if c["op"] == "decode":
            n = pgd.paged_gqa_workspace_size_ex(s["pool"], c["B"], c["q_len"], c["hq"])
            s["ws"] = torch.zeros(max(n, 256), dtype=torch.uint8, device=dev)
        elif c["op"] == "shared":
            s["ws"] = pgd.alloc_workspace_shared(s["pool"], c["B"], c["q_len"], c["hq"],
                                                 c["groups"])
    return s


def _run_own(s):
    c, pgd = s["case"], s["pgd"]
    kw = {"softcap": c["cap"], "slopes": s["slopes"], "out": s["out"]}
    if c["op"] == "attend":
        return pgd.paged_gqa_attend(s["pool"], s["q"], s["cu"], s["table"], s["lens"], s["scale"],
                                    causal=c["causal"], window=c["window"], visible=s["visible"],
                                    **kw)
    if c["op"] == "decode":
        return pgd.paged_gqa_decode_ex(s["pool"], s["q"], s["table"], s["lens"], s["scale"],
                                       window=c["window"], workspace=s["ws"], **kw)
    return pgd.paged_gqa_decode_shared(s["pool"], s["q"], s["cu_groups"], s["shared_lens"],
                                       s["table"], s["lens"], s["scale"], workspace=s["ws"], **kw)


# ------------------------------------------------------------------ plain forms

def _bits(t):
    return t.view(torch.uint8) if t.element_size() == 1 else t


def _load(s, x, blk, slot):
    """float32 values of pool `x` at the given blocks and slots."""
    pool, sc = s[x], s[x + "_scale"]
    rows = (_bits(pool)[blk, slot]).view(pool.dtype).float()
    if sc is None:
        return rows
    return rows * (sc[:, None] if s["case"]["scales"] == "head" else sc[blk][..., None])


def _tokens(s, table, t, there):
    """K and V [B, Hkv, tokens, D] of tokens t [B or 1, tokens], zeros where `there` is not."""
    bs = s["case"]["bs"]
    at = (t // bs).clamp(max=table.shape[1] - 1).expand(table.shape[0], -1)
    blk, slot = table.long().gather(1, at).clamp(min=0), t % bs
    there = there[:, :, None, None]
    return [torch.where(there, _load(s, x, blk, slot), 0.0).transpose(1, 2) for x in ("k", "v")]


def _scores(s, q, k, pos, t):
    """Shaped scores [B, Hkv, G, n, tokens] of q [B, n, Hq, D] at positions pos [B, n]."""
    c = s["case"]
    B, n = pos.shape
    group = c["hq"] // c["hkv"]
    q = q.float().view(B, n, c["hkv"], group, c["d"]).permute(0, 2, 3, 1, 4)
    p = (q.reshape(B, c["hkv"], group * n, c["d"]) * s["scale"]) @ k.transpose(2, 3)
    p = p.view(B, c["hq"], n, -1)
    if c["cap"]:
        p.div_(c["cap"]).tanh_().mul_(c["cap"])
    if s["slopes"] is not None:
        far = (pos[:, :, None] - t[:, None]).abs().float()
        p.addcmul_(far[:, None], s["slopes"][:, None, None], value=-1.0)
    return p.view(B, c["hkv"], group, n, -1)


def _softmax(p):
    """Weights, in place, and their sums; zeros where nothing is seen."""
    top = p.amax(-1, keepdim=True)
    p.sub_(torch.where(torch.isfinite(top), top, 0.0)).exp_()
    total = p.sum(-1)
    return p, torch.where(total > 0, total, 1.0)


def _values(p, v):
    """[B, n, Hq, D] of weights [B, Hkv, G, n, tokens] and v [B, Hkv, tokens, D]."""
    B, hkv, group, n, tokens = p.shape
    o = p.reshape(B, hkv, group * n, tokens) @ v
    return o.view(B, hkv, group, n, -1).permute(0, 3, 1, 2, 4).reshape(B, n, hkv * group, -1)


def _heads(total):
    """[B, Hkv, G, n] as a factor of [B, n, Hq, D]."""
    B, hkv, group, n = total.shape
    return total.permute(0, 3, 1, 2).reshape(B, n, hkv * group, 1)


def _dense(s):
    """attend and decode: scores of every sequence, padded to the longest."""
    c = s["case"]
    cu, lens = s["cu"].long(), s["lens"].long()
    n = cu[1:] - cu[:-1]
    dev = cu.device
    t = torch.arange(s["max_len"], device=dev)[None]
    i = torch.arange(s["max_new"], device=dev)
    rows = (cu[:-1, None] + i[None]).clamp(max=s["T"] - 1)            # [B, nmax]
    pos = lens[:, None] - n[:, None] + i[None]
    k, v = _tokens(s, s["table"], t, t < lens[:, None])
    p = _scores(s, s["q"].view(s["T"], c["hq"], c["d"])[rows], k, pos, t)
    see = (t < lens[:, None])[:, None].expand(-1, s["max_new"], -1)
    if c["causal"]:
        see = see & (t[:, None] <= pos[:, :, None])
        if c["window"]:
            see = see & (t[:, None] > pos[:, :, None] - c["window"])
    if s["visible"] is not None:
        ends = s["visible"].long()[rows]
        see = see & (t[:, None] >= ends[:, :, :1]) & (t[:, None] < ends[:, :, 1:])
    p.masked_fill_(~see[:, None, None], float("-inf"))
    p, total = _softmax(p)
    o = _values(p, v) / _heads(total)
    b = torch.repeat_interleave(torch.arange(c["B"], device=dev), n, output_size=s["T"])
    return o[b, torch.arange(s["T"], device=dev) - cu[b]].to(s["q"].dtype).view(s["q"].shape)


def _shared(s):
    """A group's prefix is scored once for all its queries, each sequence's own tokens alone."""
    c = s["case"]
    lens, dev, n = s["lens"].long(), s["lens"].device, c["q_len"]
    out = torch.empty_like(s["q"])
    for first, end, pre in s["groups"]:
        m = end - first
        if not m:
            continue
        q, L = s["q"][first:end], lens[first:end]
        pos = L[:, None] - n + torch.arange(n, device=dev)[None]
        t = torch.arange(pre, device=dev)[None]
        pk, pv = _tokens(s, s["table"][first:first + 1], t, t >= 0)
        a = _scores(s, q.reshape(1, m * n, c["hq"], c["d"]), pk, pos.reshape(1, -1), t)
        own_max = c["len_hi"]
        t = pre + torch.arange(own_max, device=dev)[None]
        sk, sv = _tokens(s, s["table"][first:end], t, t < L[:, None])
        b = _scores(s, q, sk, pos, t)
        see = t[:, None] <= pos[:, :, None]
        b.masked_fill_(~see[:, None, None], float("-inf"))
        hkv, group = b.shape[1:3]
        a = a.view(hkv, group, m, n, pre).permute(2, 0, 1, 3, 4)
        p, total = _softmax(torch.cat((a, b), -1))
        a, b = p[..., :pre], p[..., pre:]
        o = _values(a.permute(1, 2, 0, 3, 4).reshape(1, hkv, group, m * n, pre), pv)
        o = o.view(m, n, c["hq"], c["d"]) + _values(b, sv)
        out[first:end] = (o / _heads(total)).to(out.dtype)
    return out


def run(state):
    if own:
        return _run_own(state)
    return _shared(state) if state["case"]["op"] == "shared" else _dense(state)


# ------------------------------------------------------- 64-bit forms, head by head

def exact(case, seed):
    c = dict(case)
    lens, new = _lengths(c)
    if c["hkv"] * c["B"] > 6000:
        return None
    s = prepare(c, seed)
    dev = s["lens"].device
    seen = torch.from_numpy(_seen(c, lens, new)).to(dev)
    q = s["q"].view(s["T"], c["hq"], c["d"])
    out = torch.zeros(s["T"], c["hq"], c["d"], dtype=torch.float64, device=dev)
    group, at = c["hq"] // c["hkv"], 0
    for b, (x, n) in enumerate(zip(lens, new)):
        if not n:
            continue
        t = torch.arange(x, device=dev)
        blk, slot = s["table"][b].long()[t // c["bs"]], t % c["bs"]
        far = (torch.arange(x - n, x, device=dev)[:, None] - t[None]).abs().double()
        lo, hi = seen[at:at + n, 0], seen[at:at + n, 1]
        hide = (t[None] < lo[:, None]) | (t[None] >= hi[:, None])
        for h in range(c["hkv"]):
            k, v = [_bits(s[y])[blk, slot, h].view(s[y].dtype).double() for y in ("k", "v")]
            if s["k_scale"] is not None:
                by = [s[y][h] if c["scales"] == "head" else s[y][blk, h][:, None]
                      for y in ("k_scale", "v_scale")]
                k, v = k * by[0].double(), v * by[1].double()
            for j in range(h * group, (h + 1) * group):
                z = q[at:at + n, j].double() @ k.T * s["scale"]
                if c["cap"]:
                    e = torch.expm1(2.0 * z / c["cap"])
                    z = c["cap"] * torch.where(torch.isinf(e), 1.0, e / (e + 2.0))
                if s["slopes"] is not None:
                    z = z - s["slopes"][j].double() * far
                w = torch.softmax(z.masked_fill(hide, float("-inf")), -1)
                out[at:at + n, j] = torch.nan_to_num(w) @ v
        at += n
    return out.view(s["q"].shape)
