"""Ragged batches over a paged cache for the page operators' tests, and the bounds
their results are held to."""
import numpy as np
import torch

import paged_gqa_decode_04_gb300 as pgd
from oracle import page_ops as ref

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn,
          "int8": torch.int8}
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a step, relative


class Batch:
    """Pools, tables and lengths on `device`; `lens` cached tokens and `new` rows a
    sequence.  Slots no sequence holds are poisoned (NaN; int8: -128), and so are the
    scales of blocks no sequence holds.  `pad` rows more than the sequences own."""

    def __init__(self, lens, new, hkv=2, d=128, bs=16, pages="bf16", scales="head", seed=0,
                 pad=0, device="cuda", spare=3):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.lens, self.new, self.bs, self.hkv, self.d = list(lens), list(new), bs, hkv, d
        self.pages, dt = pages, DTYPES[pages]
        self.act = torch.float32 if pages == "f32" else torch.bfloat16
        B = len(self.lens)
        per = [-(-x // bs) for x in self.lens]
        nb = sum(per) + spare
        perm = rng.permutation(nb)
        mb = max(max(per, default=1), 1) + 1
        table = np.full((B, mb), -1, dtype=np.int32)
        at = 0
        for b in range(B):
            table[b, :per[b]] = perm[at:at + per[b]]
            at += per[b]
        shape = (nb, bs, hkv, d)
        self.k_scale = self.v_scale = None
        if dt in ref.TOP:
            top = ref.TOP[dt]
            pools = [(torch.randn(shape, generator=g) * top / 4).clamp(-top, top)
                     for _ in range(2)]
            pools = [(p.round() if dt == torch.int8 else p).to(dt) for p in pools]
            by = (nb, hkv) if scales == "block" else (hkv,)
            self.k_scale, self.v_scale = [(0.5 + torch.rand(by, generator=g)) * 4 / top
                                          for _ in range(2)]
        else:
            pools = [torch.randn(shape, generator=g).to(dt) for _ in range(2)]
        held = torch.zeros((nb, bs), dtype=torch.bool)
        for b in range(B):
            for t in range(self.lens[b]):
                held[table[b][t // bs], t % bs] = True
        for p in pools:
            bits = p.view(torch.uint8) if p.element_size() == 1 else p
            bits[~held] = {"e4m3": 0x7f, "int8": 0x80}.get(pages, float("nan"))
        if scales == "block" and self.k_scale is not None:
            for s in (self.k_scale, self.v_scale):
                s[~held.any(1)] = float("nan")
        self.k, self.v = pools
        self.table = torch.from_numpy(table)
        self.cu = torch.tensor([0] + list(np.cumsum(self.new)), dtype=torch.int32)
        self.len_t = torch.tensor(self.lens, dtype=torch.int32)
        self.total = sum(self.new) + pad
        self.g, self.device = g, device

    def rows(self, heads, scale=1.0, packed=True):
        """[total, heads, D] activations as a view of wider rows."""
        wide = torch.randn((self.total, heads + (2 if packed else 0), self.d), generator=self.g)
        return (wide * scale).to(self.act)[:, (1 if packed else 0):][:, :heads]

    def to(self, t):
        """On the device, with the strides it has here."""
        if t is None:
            return None
        base = t._base if t._base is not None else t
        moved = base.to(self.device)
        return moved.as_strided(t.shape, t.stride(), t.storage_offset())

    def pool(self):
        self.dk, self.dv = self.k.to(self.device), self.v.to(self.device)
        self.dks, self.dvs = self.to(self.k_scale), self.to(self.v_scale)
        return pgd.PagedKVPool(self.dk, self.dv, self.dks, self.dvs)

    def where(self):
        return [t.to(self.device) for t in (self.cu, self.table, self.len_t)]

    def held_rows(self):
        return [r for b in range(len(self.lens)) for r, _ in ref.rows_of(self.cu, self.lens, b)]


def bits(t):
    return t.view(torch.uint8 if t.element_size() == 1 else
                  torch.int16 if t.element_size() == 2 else torch.int32)


def check_stored(batch, which, want, size, pool_after, scale_after, slack):
    """Every element of a pool after a write: the rows stored hold `want` ({row:
    float64}) to half a step of the pages' type, plus `slack` relative to `size` for the
    float32 arithmetic before it; earlier tokens of a rescaled block moved by at most
    half a code step; everything else is as it was."""
    before = getattr(batch, which)
    scale = getattr(batch, which + "_scale")
    dt, bs = before.dtype, batch.bs
    after = pool_after.cpu()
    same = torch.ones(before.shape[:2], dtype=torch.bool)
    top = ref.TOP.get(dt)
    new_scale = scale_after.cpu() if scale is not None else None
    if scale is not None and scale.dim() == 2:
        scales = ref.block_scales(before, scale, want, batch.cu, batch.table, batch.lens)
        untouched = torch.ones(before.shape[0], dtype=torch.bool)
        for blk, s in scales.items():
            untouched[blk] = False
            # a product with a rounded reciprocal: two roundings, and the rows' own error
            assert torch.all((new_scale[blk].double() - s).abs() <= s * (2.0 ** -23 + slack)), blk
        assert torch.equal(bits(new_scale[untouched]), bits(scale[untouched]))
    elif scale is not None:
        assert torch.equal(new_scale, scale)
    for b in range(len(batch.lens)):
        todo = ref.rows_of(batch.cu, batch.lens, b)
        if not todo:
            continue
        for row, pos in todo:
            blk, slot = ref.place(batch.table, bs, b, pos)
            same[blk, slot] = False
            got, y, m = after[blk, slot].double(), want[row], size[row]
            if top is None:
                assert torch.all((got - y).abs() <= ROUND[dt] * y.abs() + slack * m), (b, pos)
                continue
            s = (new_scale if scale.dim() == 1 else new_scale[blk]).double()[:, None]
            inv = torch.where(s > 0, 1 / s, 0.0)
            z = (y * inv).clamp(-top, top)
            err = (got - z).abs() - ref.half_step(z, dt)
            assert torch.all(err <= (slack + 2.0 ** -22) * m * inv), (b, pos)
        first = todo[0][1]
        if scale is not None and scale.dim() == 2 and first % bs:
            blk = int(batch.table[b][first // bs])
            ratio = (scale[blk].double() / new_scale[blk].double().clamp(min=2.0 ** -126))[:, None]
            for slot in range(first % bs):
                same[blk, slot] = False
                z = before[blk, slot].double() * torch.minimum(ratio, torch.ones_like(ratio))
                err = (after[blk, slot].double() - z).abs()
                moved = (ratio < 1) * (ref.half_step(z, dt) * (1 + 2.0 ** -20) + 2.0 ** -20)
                assert torch.all(err <= moved), (b, slot)
    assert torch.equal(bits(after)[same], bits(before)[same])
