// paged_gqa_decode_shared: decode of sequences that share prefixes in groups.
// See include/paged_gqa.h for the contract.
//
// A query's softmax over its tokens [0, L) is that over [0, S) joined with that over [S, L),
//     out = (2^a o_0 + 2^b o_1) / (2^a + 2^b),   a, b the base-2 log-sum-exp of the scores.
// Three kernels, one after the other:
//   1. the attention kernel of attend_tc.cuh over a group's first S tokens, for the queries of
//      all its sequences at once: with many sequences a product of matrices, and each page of
//      the prefix comes once for every 256 query rows instead of once a sequence.  Its keys are
//      cut into parts for as many CTAs as the GPU holds (prefix_splits, prefix_parts), each of
//      which leaves (o, lse) of its rows; one CTA more writes S of every sequence;
//   2. the decode kernel over every sequence's tokens from S on;
//   3. the join of both, a row's parts at a time (join_kernel).
#include "attend_launch.cuh"
#include "page_ops.h"
#include "ragged.cuh"

namespace pgd {
namespace {

// Workspace after the decode's own.
struct SharedLayout {
    size_t starts_off, row_lse_off, row_o_off, pre_lse_off, pre_o_off, total;
    int splits;
};

SharedLayout shared_layout(const Pool& p, size_t decode_bytes, int B, int q_len, int Hq,
                           int groups) {
    SharedLayout w;
    const size_t rows = (size_t)B * q_len * Hq;
    w.splits = groups > 0 ? attend::prefix_splits((int64_t)B * q_len * (Hq / p.hkv), groups,
                                                  p.hkv, p.num_sms)
                          : 0;
    w.starts_off = round_up(decode_bytes, 256);
    w.row_lse_off = w.starts_off + round_up((size_t)B * sizeof(int32_t), 256);
    w.row_o_off = w.row_lse_off + round_up(rows * sizeof(float), 256);
    w.pre_lse_off = w.row_o_off + round_up(rows * p.d * sizeof(float), 256);
    const size_t most = groups > 0 ? attend::most_prefix_rows(rows, p.num_sms) : 0;
    w.pre_o_off = w.pre_lse_off + round_up(most * sizeof(float), 256);
    w.total = w.pre_o_off + round_up(most * p.d * sizeof(float), 256);
    return w;
}

}  // namespace
}  // namespace pgd

using namespace pgd;

extern "C" int paged_gqa_workspace_size_shared(pgd_pool_t pool, int B, int q_len, int Hq,
                                               int num_groups, size_t* bytes) {
    size_t decode = 0;
    if (num_groups < 0 || !bytes) return PGD_ERR_ARG;
    const int rc = paged_gqa_workspace_size_ex(pool, B, q_len, Hq, 0, &decode);
    if (rc != PGD_OK) return rc;
    *bytes = shared_layout(pool_desc(pool), decode, B, q_len, Hq, num_groups).total;
    return PGD_OK;
}

extern "C" int paged_gqa_decode_shared(pgd_pool_t pool, const void* q, int B, int q_len, int Hq,
                                       const int32_t* cu_groups, const int32_t* shared_lens,
                                       int num_groups, const int32_t* block_table, int max_blocks,
                                       const int32_t* seq_lens, float scale, float softcap,
                                       const float* slopes, void* out, void* workspace,
                                       size_t workspace_bytes, void* stream) {
    if (!pool || num_groups < 0) return PGD_ERR_ARG;
    const float scale_log2 = fabsf(scale) * kLog2e;
    if (!isfinite(scale_log2)) return PGD_ERR_ARG;
    int rc = check_shaping(softcap, slopes);
    if (rc != PGD_OK) return rc;
    const Pool& p = pool_desc(pool);
    if (p.dtype == PGD_F32) return PGD_ERR_UNSUPPORTED;
    Plan plan;
    WorkspaceLayout wl;
    rc = check_decode(p, q, B, q_len, Hq, block_table, max_blocks, seq_lens, 0, scale, out,
                      workspace, workspace_bytes, 0, &plan, &wl);
    if (rc != PGD_OK || B == 0) return rc;
    // token positions plus a tile stay within 31 bits
    if ((int64_t)max_blocks * p.block_size > INT32_MAX - 1024) return PGD_ERR_SHAPE;
    if (num_groups > 0) {
        if (!cu_groups || !shared_lens) return PGD_ERR_ARG;
        if (!is_aligned(cu_groups, 4) || !is_aligned(shared_lens, 4)) return PGD_ERR_ALIGN;
    }
    SharedLayout sl = shared_layout(p, wl.total, B, q_len, Hq, num_groups);
    if (workspace_bytes < sl.total) return PGD_ERR_WORKSPACE;
    // at the end, so that a decode of more sequences finds its counters as it left them
    const size_t by = workspace_bytes / 256 * 256 - sl.total;
    place_at_end(&wl, wl.total + by);
    for (size_t* off : {&sl.starts_off, &sl.row_lse_off, &sl.row_o_off, &sl.pre_lse_off,
                        &sl.pre_o_off})
        *off += by;
    const int group = Hq / p.hkv, per = group * q_len;
    const int64_t pieces = max_pieces(B, num_groups, per, attend::kRowShift, 1);
    if ((int64_t)B * q_len * Hq > INT32_MAX / 2) return PGD_ERR_SHAPE;
    if (pieces * p.hkv * (sl.splits + 1) > INT32_MAX - 1) return PGD_ERR_SHAPE;
    OnDevice dev(p.device);
    if (!dev.ok) return PGD_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    DecodeArgs a = decode_args(p, q, B, q_len, Hq, block_table, max_blocks, seq_lens, 0, scale,
                               softcap, slopes, out, workspace, 0, plan, wl);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.join = 1;
    a.row_lse = reinterpret_cast<float*>(ws + sl.row_lse_off);
    a.row_o = reinterpret_cast<float*>(ws + sl.row_o_off);
    if (num_groups > 0) {
        int32_t* const starts = reinterpret_cast<int32_t*>(ws + sl.starts_off);
        attend::Args t = {};
        t.r = {cu_groups, block_table, seq_lens, num_groups, B * q_len, max_blocks, p.block_size,
               p.num_blocks, max_blocks * p.block_size, p.err};
        t.hq = Hq;
        t.hkv = p.hkv;
        t.group = group;
        t.q = static_cast<const __nv_bfloat16*>(q);
        t.q_stride = (int64_t)Hq * p.d;
        t.scale_log2 = scale != 0.f ? scale_log2 : 1.f;
        t.q_and = scale != 0.f ? 0xffffffffu : 0u;
        t.q_xor = scale < 0.f ? 0x80008000u : 0u;
        t.pieces = int(pieces);
        t.k_scale = p.k_scale;
        t.v_scale = p.v_scale;
        attend::set_cap(t, a.cap);
        t.slopes = slopes;
        t.shared = shared_lens;
        t.starts = starts;
        t.batch = B;
        t.q_len = q_len;
        t.splits = sl.splits;
        t.part_o = reinterpret_cast<float*>(ws + sl.pre_o_off);
        t.part_lse = reinterpret_cast<float*>(ws + sl.pre_lse_off);
        if (attend::launch_attend(t, p, page_maps(pool), true, s) != cudaSuccess)
            return PGD_ERR_CUDA;
        a.starts = starts;
        a.prefix_splits = sl.splits;
        a.pre_o = t.part_o;
        a.pre_lse = t.part_lse;
    }
    if (launch_decode_ex(a, p, s) != cudaSuccess) return PGD_ERR_CUDA;
    return launch_join(a, s) == cudaSuccess ? PGD_OK : PGD_ERR_CUDA;
}
