"""Python face of the KV write path (include/paged_kv_manager.h).

``KVBlockManager`` wraps the C++ host block manager (on-demand block
allocation, reference counts, copy-on-write of a shared last block);
``paged_kv_append`` and ``paged_kv_copy_blocks`` wrap the device kernels that
store new tokens and copy blocks; ``paged_kv_write``, ``paged_kv_read`` and
``paged_qk_norm_rope_write`` those of ragged batches (quantising, reading back,
norm and rotation with the write).  Argument marshalling only.
"""
import ctypes

import numpy as np
import torch

from . import _lib
from ._lib import PagedGQAError


def _check(rc, what=""):
    if rc != 0:
        raise PagedGQAError(rc, what)


def _ints(seqs):
    arr = (ctypes.c_int * len(seqs))(*[int(s) for s in seqs])
    return arr


class KVBlockManager:
    """Host-side owner of a pool's blocks: which sequence holds which blocks."""

    def __init__(self, num_blocks, block_size, max_seqs, max_blocks_per_seq):
        lib = _lib.load()
        h = ctypes.c_void_p()
        _check(lib.pgd_kvm_create(ctypes.byref(h), int(num_blocks), int(block_size),
                                  int(max_seqs), int(max_blocks_per_seq)), "pgd_kvm_create")
        self._h = h
        self.block_size = int(block_size)
        self.max_blocks_per_seq = int(max_blocks_per_seq)

    def close(self):
        if getattr(self, "_h", None) is not None and _lib._lib is not None:
            _lib._lib.pgd_kvm_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def add_sequence(self, seq):
        _check(_lib.load().pgd_kvm_add_sequence(self._h, int(seq)), "add_sequence")

    def fork(self, parent, child):
        _check(_lib.load().pgd_kvm_fork(self._h, int(parent), int(child)), "fork")

    def free_sequence(self, seq):
        _check(_lib.load().pgd_kvm_free_sequence(self._h, int(seq)), "free_sequence")

    def append_slots(self, seqs):
        """Reserve one new token position per sequence.  Returns (slots int32
        array, [(src_block, dst_block), ...] copies to run first)."""
        n = len(seqs)
        slots = np.empty(n, dtype=np.int32)
        src = np.empty(max(n, 1), dtype=np.int32)
        dst = np.empty(max(n, 1), dtype=np.int32)
        nc = ctypes.c_int()
        p32 = ctypes.POINTER(ctypes.c_int32)
        _check(_lib.load().pgd_kvm_append_slots(
            self._h, _ints(seqs), n, slots.ctypes.data_as(p32), src.ctypes.data_as(p32),
            dst.ctypes.data_as(p32), ctypes.byref(nc)), "append_slots")
        return slots, list(zip(src[:nc.value].tolist(), dst[:nc.value].tolist()))

    def block_tables(self, seqs, max_blocks=None):
        """(table [n, max_blocks] int32 with -1 past each sequence's blocks, lens [n] int32)."""
        max_blocks = int(max_blocks or self.max_blocks_per_seq)
        n = len(seqs)
        table = np.empty((n, max_blocks), dtype=np.int32)
        lens = np.empty(n, dtype=np.int32)
        p32 = ctypes.POINTER(ctypes.c_int32)
        _check(_lib.load().pgd_kvm_block_tables(self._h, _ints(seqs), n, table.ctypes.data_as(p32),
                                                max_blocks, lens.ctypes.data_as(p32)),
               "block_tables")
        return table, lens

    def num_free(self):
        n = ctypes.c_int64()
        _check(_lib.load().pgd_kvm_num_free(self._h, ctypes.byref(n)))
        return n.value

    def ref_count(self, block):
        c = ctypes.c_int()
        _check(_lib.load().pgd_kvm_ref_count(self._h, int(block), ctypes.byref(c)))
        return c.value


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if isinstance(stream, torch.cuda.Stream)
                           else int(stream))


def paged_kv_append(pool, k_new, v_new, slot_mapping, stream=None):
    """Store n new tokens: k_new / v_new [n, Hkv, D] (pool dtype, CUDA),
    slot_mapping [n] int32 CUDA tensor of physical slots."""
    if k_new.shape != v_new.shape or k_new.dim() != 3 or k_new.dtype != pool.dtype:
        raise ValueError("k_new / v_new must be [n, Hkv, D] in the pool's dtype (8-bit codes "
                         "for 8-bit pools, already scaled)")
    if slot_mapping.dtype != torch.int32 or slot_mapping.numel() != k_new.shape[0]:
        raise ValueError("slot_mapping must be int32 with one slot per new token")
    for t in (k_new, v_new, slot_mapping):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("inputs must be contiguous CUDA tensors")
    _check(_lib.load().paged_kv_append(pool.handle, k_new.data_ptr(), v_new.data_ptr(),
                                       slot_mapping.data_ptr(), k_new.shape[0], _stream(stream)),
           "paged_kv_append")


def paged_kv_copy_blocks(pool, src, dst, stream=None):
    """Copy whole blocks src[i] -> dst[i] (int32 CUDA tensors), K and V."""
    if src.dtype != torch.int32 or dst.dtype != torch.int32 or src.shape != dst.shape:
        raise ValueError("src and dst must be int32 tensors of one shape")
    _check(_lib.load().paged_kv_copy_blocks(pool.handle, src.data_ptr(), dst.data_ptr(),
                                            src.numel(), _stream(stream)), "paged_kv_copy_blocks")


def _check_tables(pool, cu_seqlens, block_table, seq_lens):
    """The tables of a ragged call: dtypes, shapes and placement.  Returns B."""
    dev, i32 = pool.device.index, torch.int32
    if cu_seqlens.dim() != 1 or block_table.dim() != 2 or seq_lens.dim() != 1:
        raise ValueError("cu_seqlens must be [B+1], block_table [B,max_blocks], seq_lens [B]")
    if not (cu_seqlens.dtype is i32 and block_table.dtype is i32 and seq_lens.dtype is i32):
        raise TypeError("cu_seqlens, block_table and seq_lens must be int32")
    B = seq_lens.shape[0]
    if cu_seqlens.shape[0] != B + 1 or block_table.shape[0] != B:
        raise ValueError("shape mismatch between cu_seqlens, block_table and seq_lens")
    if B >= 2 ** 31 or block_table.shape[1] >= 2 ** 31:   # the library takes them as C ints
        raise ValueError("block_table must have fewer than 2^31 rows and columns")
    for t in (cu_seqlens, block_table, seq_lens):
        if t.get_device() != dev or not t.is_contiguous():   # -1 for CPU tensors
            raise ValueError("tables must be contiguous CUDA tensors on the pool's device")
    return B


def _check_rows(pool, name, t, heads, total=None):
    """A packed tensor [total, heads, D] whose rows may be apart (a view of a
    projection); returns its row stride in elements."""
    shape, D = t.shape, pool.head_dim
    if len(shape) != 3 or shape[1] != heads or shape[2] != D or (
            total is not None and shape[0] != total):
        raise ValueError("%s must be [total, %s, %d]" % (name, heads, D))
    if t.dtype is not pool.q_dtype:
        raise TypeError("%s must be %s for this pool" % (name, pool.q_dtype))
    if t.get_device() != pool.device.index:
        raise ValueError("%s must be a CUDA tensor on the pool's device" % name)
    if shape[0] == 0 or heads == 0:
        return heads * D
    s0, s1, s2 = t.stride()
    if s2 != 1 or (heads > 1 and s1 != D):
        raise ValueError("%s: the heads of a row must be contiguous" % name)
    return s0 if shape[0] > 1 else heads * D


def _stream_on(pool, stream):
    """The stream to launch on: by default the current one of the pool's device."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(pool.device.index)
    return _stream(stream)


def _empty_on(pool, stream, shape):
    """An output allocated on the launching stream, so that its memory is not handed
    out again before the launch is done with it."""
    if stream is None:
        return torch.empty(shape, dtype=pool.q_dtype, device=pool.device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=pool.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=pool.q_dtype, device=pool.device)


def _zeros_on(pool, stream, nbytes):
    """A zero-filled workspace allocated and cleared on the launching stream."""
    if stream is None:
        return torch.zeros(nbytes, dtype=torch.uint8, device=pool.device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=pool.device)
    with torch.cuda.stream(stream):
        return torch.zeros(nbytes, dtype=torch.uint8, device=pool.device)


def paged_kv_write(pool, k, v, cu_seqlens, block_table, seq_lens, stream=None):
    """Store the new tokens of a ragged batch in the pages, quantised as they are
    written.

    k, v [total, Hkv, D] (bfloat16; float32 for float32 pools; rows may be a view of a
    packed projection): rows cu_seqlens[b] .. cu_seqlens[b+1]-1 are the last ones of
    the seq_lens[b] cached tokens of sequence b.  8-bit pools with a scale per block
    have the scales of the written blocks set (see paged_kv_manager.h).
    """
    B = _check_tables(pool, cu_seqlens, block_table, seq_lens)
    ks = _check_rows(pool, "k", k, pool.num_kv_heads)
    vs = _check_rows(pool, "v", v, pool.num_kv_heads, k.shape[0])
    _check(_lib.load().paged_kv_write(
        pool.handle, k.data_ptr(), ks, v.data_ptr(), vs, k.shape[0], cu_seqlens.data_ptr(), B,
        block_table.data_ptr(), block_table.shape[1], seq_lens.data_ptr(),
        _stream_on(pool, stream)), "paged_kv_write")


def paged_kv_read(pool, total, cu_seqlens, block_table, seq_lens, out=None, stream=None):
    """Read the last cu_seqlens[b+1] - cu_seqlens[b] cached tokens of every sequence
    back as packed rows (k, v), [total, Hkv, D] each, dequantised.  `out`: the pair to
    write into; rows past cu_seqlens[B] are left as they were."""
    B = _check_tables(pool, cu_seqlens, block_table, seq_lens)
    total = int(total)
    if total < 0:
        raise ValueError("total must not be negative")
    shape = (total, pool.num_kv_heads, pool.head_dim)
    if out is None:
        out = (_empty_on(pool, stream, shape), _empty_on(pool, stream, shape))
    k_out, v_out = out
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        _check_rows(pool, name, t, pool.num_kv_heads, total)
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)
    _check(_lib.load().paged_kv_read(
        pool.handle, k_out.data_ptr(), v_out.data_ptr(), total, cu_seqlens.data_ptr(), B,
        block_table.data_ptr(), block_table.shape[1], seq_lens.data_ptr(),
        _stream_on(pool, stream)), "paged_kv_read")
    return k_out, v_out


def rope_table(length, rope_dim, base=10000.0, device=None):
    """Rotation table [length, 2, rope_dim / 2] float32 for paged_qk_norm_rope_write:
    cosines and sines of p * base^(-2j / rope_dim), computed in float64."""
    half = int(rope_dim) // 2
    j = torch.arange(half, dtype=torch.float64, device=device)
    angle = torch.arange(int(length), dtype=torch.float64, device=device)[:, None] * (
        float(base) ** (-j / half))
    return torch.stack((angle.cos(), angle.sin()), 1).float()


def _check_weight(pool, name, w):
    if w is None:
        return None
    if w.dim() != 1 or w.shape[0] != pool.head_dim or not w.is_contiguous():
        raise ValueError("%s must be a contiguous [%d]" % (name, pool.head_dim))
    if w.dtype is not torch.float32 and w.dtype is not torch.bfloat16:
        raise TypeError("%s must be float32 or bfloat16" % name)
    if w.get_device() != pool.device.index:
        raise ValueError("%s must be on the pool's device" % name)
    return w.data_ptr()


def paged_qk_norm_rope_write(pool, q, k, v, cu_seqlens, block_table, seq_lens, q_weight=None,
                             k_weight=None, eps=1e-6, rope=None, interleaved=False, q_out=None,
                             stream=None):
    """Norm each head of q and k (q_weight, k_weight [D], None: no norm), rotate them by
    position (rope [positions, 2, rope_dim / 2], see rope_table; None: no rotation),
    and store k and v in the pages as paged_kv_write does, in one pass.  Returns q_out
    [total, Hq, D], which may be q itself."""
    B = _check_tables(pool, cu_seqlens, block_table, seq_lens)
    if q.dim() != 3:
        raise ValueError("q must be [total, Hq, D]")
    total, Hq = q.shape[0], q.shape[1]
    qs = _check_rows(pool, "q", q, Hq)
    ks = _check_rows(pool, "k", k, pool.num_kv_heads, total)
    vs = _check_rows(pool, "v", v, pool.num_kv_heads, total)
    qw, kw = _check_weight(pool, "q_weight", q_weight), _check_weight(pool, "k_weight", k_weight)
    if qw and kw and q_weight.dtype is not k_weight.dtype:
        raise TypeError("q_weight and k_weight must share one dtype")
    given = q_weight if q_weight is not None else k_weight
    w_code = _lib.PGD_F32 if given is not None and given.dtype == torch.float32 else _lib.PGD_BF16
    r_ptr, r_len, r_dim = None, 0, 0
    if rope is not None:
        if rope.dim() != 3 or rope.shape[1] != 2 or rope.dtype is not torch.float32:
            raise ValueError("rope must be float32 [positions, 2, rope_dim / 2]")
        if not rope.is_contiguous() or rope.get_device() != pool.device.index:
            raise ValueError("rope must be contiguous and on the pool's device")
        r_ptr, r_len, r_dim = rope.data_ptr(), rope.shape[0], 2 * rope.shape[2]
    if q_out is None:
        q_out = _empty_on(pool, stream, tuple(q.shape))
    os_ = _check_rows(pool, "q_out", q_out, Hq, total)
    _check(_lib.load().paged_qk_norm_rope_write(
        pool.handle, q.data_ptr(), qs, q_out.data_ptr(), os_, Hq, k.data_ptr(), ks, v.data_ptr(),
        vs, total, qw, kw, w_code, float(eps), r_ptr, r_len, r_dim, int(bool(interleaved)),
        cu_seqlens.data_ptr(), B, block_table.data_ptr(), block_table.shape[1],
        seq_lens.data_ptr(), _stream_on(pool, stream)), "paged_qk_norm_rope_write")
    return q_out


def _slopes_ptr(pool, slopes, heads):
    """The pointer of distance slopes [Hq], or None."""
    if slopes is None:
        return None
    if slopes.dim() != 1 or slopes.shape[0] != heads or not slopes.is_contiguous():
        raise ValueError("slopes must be a contiguous [%d]" % heads)
    if slopes.dtype is not torch.float32:
        raise TypeError("slopes must be float32")
    if slopes.get_device() != pool.device.index:
        raise ValueError("slopes must be on the pool's device")
    return slopes.data_ptr() if heads else None


def paged_gqa_attend(pool, q, cu_seqlens, block_table, seq_lens, scale, causal=True, window=0,
                     out=None, stream=None, softcap=0.0, slopes=None, visible=None):
    """Attention of a ragged batch of query tokens over the pages.

    q [total, Hq, D] bfloat16 (rows may be a view of a packed projection): rows
    cu_seqlens[b] .. cu_seqlens[b+1]-1 belong to sequence b.  causal: they are its last
    cached tokens and attend to what comes before them (the `window` most recent
    tokens when window > 0): prompts and chunks of prompts.  Not causal: every query
    attends to all seq_lens[b] cached tokens: cross attention.  Returns out
    [total, Hq, D]; rows past cu_seqlens[B] are left as they were.  Sums are float32, the
    weights that V is multiplied with bfloat16 (f16 over 8-bit pages, see paged_gqa.h).

    Shaped scores: softcap > 0 takes s to softcap * tanh(s / softcap); slopes [Hq] float32
    then subtract slopes[h] * |p - t| (query i of n at p = seq_lens[b] - n + i); visible
    [total, 2] int32 lets a row see tokens [first, end) alone, of those it would see without
    (packed documents; with causal=False a prefix that all rows see: [0, max(p + 1, prefix))).
    """
    B = _check_tables(pool, cu_seqlens, block_table, seq_lens)
    if q.dim() != 3:
        raise ValueError("q must be [total, Hq, D]")
    total, Hq = q.shape[0], q.shape[1]
    qs = _check_rows(pool, "q", q, Hq)
    if out is None:
        out = _empty_on(pool, stream, tuple(q.shape))
    _check_rows(pool, "out", out, Hq, total)
    if not out.is_contiguous():
        raise ValueError("out must be contiguous")
    window = min(max(int(window), -1), 2 ** 31 - 1)   # none there is longer; C takes an int
    v_ptr = None
    if visible is not None:
        if visible.dim() != 2 or tuple(visible.shape) != (total, 2) or \
                not visible.is_contiguous():
            raise ValueError("visible must be a contiguous [total, 2]")
        if visible.dtype is not torch.int32:
            raise TypeError("visible must be int32")
        if visible.get_device() != pool.device.index:
            raise ValueError("visible must be on the pool's device")
        v_ptr = visible.data_ptr() if total else None
    _check(_lib.load().paged_gqa_attend_shaped(
        pool.handle, q.data_ptr(), qs, total, Hq, cu_seqlens.data_ptr(), B,
        block_table.data_ptr(), block_table.shape[1], seq_lens.data_ptr(), int(bool(causal)),
        window, float(scale), float(softcap), _slopes_ptr(pool, slopes, Hq), v_ptr,
        out.data_ptr(), _stream_on(pool, stream)), "paged_gqa_attend")
    return out


def paged_gqa_workspace_size_shared(pool, B, q_len, Hq, num_groups):
    n = ctypes.c_size_t()
    _check(_lib.load().paged_gqa_workspace_size_shared(
        pool.handle, int(B), int(q_len), int(Hq), int(num_groups), ctypes.byref(n)),
        "paged_gqa_workspace_size_shared")
    return n.value


def alloc_workspace_shared(pool, B, q_len, Hq, num_groups):
    """A zero-filled workspace for paged_gqa_decode_shared, reusable call after call."""
    n = paged_gqa_workspace_size_shared(pool, B, q_len, Hq, num_groups)
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=pool.device)


def paged_gqa_decode_shared(pool, q, cu_groups, shared_lens, block_table, seq_lens, scale,
                            softcap=0.0, slopes=None, out=None, workspace=None, stream=None):
    """Decode of sequences that share prefixes in groups, as forks of one prompt do.

    q [B, Hq, D] or [B, q_len, Hq, D] bfloat16: the last tokens of each sequence, as for
    paged_gqa_decode_ex.  Sequences cu_groups[g] .. cu_groups[g+1]-1 (int32 [groups + 1])
    are group g; their first shared_lens[g] (int32 [groups]) cached tokens are the same, and
    are read once for the group, through the table row of one of its sequences.  softcap and
    slopes as for paged_gqa_attend.  Returns out, shaped like q.
    """
    if q.dim() not in (3, 4):
        raise ValueError("q must be [B, Hq, D] or [B, q_len, Hq, D]")
    if q.dtype is not pool.q_dtype:
        raise TypeError("q must be %s for this pool" % pool.q_dtype)
    B, Hq, q_len = q.shape[0], q.shape[-2], q.shape[1] if q.dim() == 4 else 1
    for name, t, dims in (("cu_groups", cu_groups, 1), ("shared_lens", shared_lens, 1),
                          ("block_table", block_table, 2), ("seq_lens", seq_lens, 1)):
        if t.dim() != dims or t.dtype is not torch.int32 or not t.is_contiguous():
            raise ValueError("%s must be a contiguous int32 tensor of %d dimensions"
                             % (name, dims))
    groups = shared_lens.shape[0]
    if (q.shape[-1] != pool.head_dim or cu_groups.shape[0] != groups + 1 or
            block_table.shape[0] != B or seq_lens.shape[0] != B):
        raise ValueError("shape mismatch between q, groups, tables and pool")
    if out is None:
        out = _empty_on(pool, stream, tuple(q.shape))
    if out.shape != q.shape or out.dtype is not q.dtype:
        raise ValueError("out must be shaped and typed like q")
    for t in (q, out, cu_groups, shared_lens, block_table, seq_lens):
        if t.get_device() != pool.device.index or not t.is_contiguous():
            raise ValueError("tensors must be contiguous and on the pool's device")
    sl = _slopes_ptr(pool, slopes, Hq)
    if workspace is None:
        workspace = _zeros_on(pool, stream, max(paged_gqa_workspace_size_shared(
            pool, B, q_len, Hq, groups), 256))
    if workspace.get_device() != pool.device.index or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on the pool's device")
    _check(_lib.load().paged_gqa_decode_shared(
        pool.handle, q.data_ptr(), B, q_len, Hq, cu_groups.data_ptr(), shared_lens.data_ptr(),
        groups, block_table.data_ptr(), block_table.shape[1], seq_lens.data_ptr(), float(scale),
        float(softcap), sl, out.data_ptr(), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream_on(pool, stream)),
        "paged_gqa_decode_shared")
    return out
