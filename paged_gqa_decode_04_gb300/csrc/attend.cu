// paged_gqa_attend: attention of a ragged batch of query tokens over the pages,
// causal (prompts, chunks of prompts) or over all cached tokens (cross attention).
// See include/paged_gqa.h for the contract.
//
//     out = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale <q, k_t> - m), m = max_t,
//
// in one pass over the tokens with a running maximum and sum in float32.  bfloat16 pools
// take the tensor-core kernel (attend_tc.cuh), 8-bit pools one warp per (query token,
// query head), a lane holding D / 32 elements.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <atomic>

#include "attend_tc.cuh"
#include "page_maps.h"
#include "page_ops.h"
#include "ragged.cuh"

namespace pgd {
namespace {

constexpr int kWarps = 8;

struct AttendArgs {
    Ragged r;
    const void* k_pool;
    const void* v_pool;
    const float* k_scale;
    const float* v_scale;
    int scale_per_block;
    int hq, hkv;
    const __nv_bfloat16* q;
    int64_t q_stride;
    __nv_bfloat16* out;
    int causal;
    int window;
    float scale_log2;
};

// D / 32 consecutive elements of a page row, element e of the pool.
template <int PAGE, int N>
__device__ __forceinline__ void page_values(const void* pool, int64_t e, float (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (PAGE == PGD_BF16)
            x[i] = __bfloat162float(static_cast<const __nv_bfloat16*>(pool)[e + i]);
        else if (PAGE == PGD_INT8)
            x[i] = float(static_cast<const int8_t*>(pool)[e + i]);
        else
            x[i] = float(static_cast<const __nv_fp8_e4m3*>(pool)[e + i]);
    }
}

template <int PAGE, int D>
__global__ void __launch_bounds__(kWarps * 32) attend_simple_kernel(const AttendArgs a) {
    constexpr int N = D / 32;
    constexpr bool q8 = PAGE != PGD_BF16;
    if (blockIdx.x == 0) check_all(a.r, false);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t unit = (int64_t)blockIdx.x * kWarps + warp;
    const int64_t t = unit / a.hq;
    const int h = int(unit % a.hq), kv = h / (a.hq / a.hkv);
    if (t >= a.r.total) return;
    const int b = find_seq(a.r, t, 1, 0, 0);
    if (b >= a.r.B) return;
    const Seq s = load_seq(a.r, b);
    if (t < s.row0 || (s.ok && t >= s.row0 + s.n)) return;
    const int pos = s.len - s.n + int(t - s.row0);  // the query's position
    int lo = 0, hi = s.len;
    if (a.causal) {
        hi = pos + 1;
        if (a.window > 0) lo = max(0, pos - a.window + 1);
    }
    float q[N], o[N], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        q[i] = __bfloat162float(a.q[t * a.q_stride + h * D + lane * N + i]);
        o[i] = 0.f;
    }
    bool bad = !s.ok;
    for (int u = lo; u < hi && !bad; ++u) {
        const int64_t blk = block_of(a.r, b, u / a.r.block_size);
        if (blk < 0) {
            bad = true;
            break;
        }
        const int64_t e = ((blk * a.r.block_size + u % a.r.block_size) * a.hkv + kv) * D + lane * N;
        float x[N];
        page_values<PAGE, N>(a.k_pool, e, x);
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) z = fmaf(q[i], x[i], z);
#pragma unroll
        for (int k = 1; k < 32; k *= 2) z += __shfl_xor_sync(0xffffffffu, z, k);
        float vs = 1.f;
        z *= a.scale_log2;
        if (q8) {
            const int64_t si = kv + (a.scale_per_block ? blk * a.hkv : 0);
            z *= a.k_scale[si];
            vs = a.v_scale[si];
        }
        const float top = fmaxf(m, z);
        const float keep = top == -INFINITY ? 1.f : exp2f(m - top);
        const float p = top == -INFINITY ? 0.f : exp2f(z - top);
        m = top;
        l = l * keep + p;
        page_values<PAGE, N>(a.v_pool, e, x);
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = fmaf(p * vs, x[i], o[i] * keep);
    }
    const float inv = bad ? NAN : l > 0.f ? 1.f / l : l == 0.f ? 0.f : NAN;
#pragma unroll
    for (int i = 0; i < N; ++i)
        a.out[(t * a.hq + h) * D + lane * N + i] =
            __float2bfloat16(inv == 0.f ? 0.f : o[i] * inv);
}

// CTAs that share the keys of a piece of rows (a cluster).  One CTA fits on an SM, so
// `units` pieces take ceil(units c / SMs) rounds of 1 / c of the work each; c is raised
// while that saves a tenth or more.  Joining the sums costs a CTA some 5 us, so each keeps
// tiles of the longest sequence that the table can hold for it: 2 where SMs are idle
// without it, 64 (about 100 us) where they only end unevenly.
int choose_cluster(const Pool& p, int64_t units, int64_t max_tokens) {
    auto rounds = [&](int c) { return double((units * c + p.num_sms - 1) / p.num_sms) / c; };
    int best = 1;
    for (int c = 2; c <= 8; c *= 2) {
        const int keep = units * c <= p.num_sms ? 2 : 64;
        if (max_tokens >= (int64_t)c * keep * attend::kTile && rounds(c) <= 0.9 * rounds(best))
            best = c;
    }
    return best;
}

template <int D>
cudaError_t launch_tc(const attend::Args& a, const Pool& p, const PageMaps& maps, cudaStream_t s) {
    using namespace attend;
    static std::atomic<uint64_t> ready{0};  // devices whose function attributes are set
    if (!(ready.load() >> p.device & 1)) {
        const cudaError_t e = cudaFuncSetAttribute(
            attend_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<D>::kBytes);
        if (e != cudaSuccess) return e;
        ready.fetch_or(uint64_t(1) << p.device);
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = a.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(unsigned(a.pieces) * a.hkv * a.cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Layout<D>::kBytes;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = a.cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, attend_kernel<D>, a, maps.k, maps.v);
}

}  // namespace
}  // namespace pgd

using namespace pgd;

extern "C" int paged_gqa_attend(pgd_pool_t pool, const void* q, int64_t q_stride, int total,
                                int Hq, const int32_t* cu_seqlens, int B,
                                const int32_t* block_table, int max_blocks,
                                const int32_t* seq_lens, int causal, int window, float scale,
                                void* out, void* stream) {
    if (!pool || Hq < 1 || window < 0 || (causal != 0 && causal != 1) || !isfinite(scale))
        return PGD_ERR_ARG;
    if (window > 0 && !causal) return PGD_ERR_ARG;
    const Pool& p = pool_desc(pool);
    if (Hq % p.hkv != 0) return PGD_ERR_SHAPE;
    if (p.dtype == PGD_F32) return PGD_ERR_UNSUPPORTED;
    int rc = check_ragged(p, total, cu_seqlens, B, block_table, max_blocks, seq_lens);
    if (rc != PGD_OK || B == 0 || total == 0) return rc;
    const int64_t width = (int64_t)Hq * p.d;
    rc = check_rows(q, q_stride, width, 2);
    if (rc == PGD_OK) rc = check_rows(out, width, width, 2);
    if (rc != PGD_OK) return rc;
    {
        const char* q0 = static_cast<const char*>(q);
        const char* o0 = static_cast<char*>(out);
        if (q0 < o0 + width * 2 * total && o0 < q0 + (q_stride * (total - 1) + width) * 2)
            return PGD_ERR_ARG;  // out aliases q
    }
    const int cap = max_blocks * p.block_size;
    const int group = Hq / p.hkv;
    if ((int64_t)total * group > INT32_MAX / 2) return PGD_ERR_SHAPE;
    const int64_t pieces = max_pieces(total, B, group, attend::kRowShift, 1);
    if (pieces * p.hkv * 8 > INT32_MAX) return PGD_ERR_SHAPE;
    OnDevice dev(p.device);
    if (!dev.ok) return PGD_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p.dtype == PGD_BF16) {
        attend::Args t = {};
        t.r = {cu_seqlens, block_table, seq_lens, B, total, max_blocks, p.block_size,
               p.num_blocks, cap, p.err};
        t.hq = Hq;
        t.hkv = p.hkv;
        t.group = group;
        t.q = static_cast<const __nv_bfloat16*>(q);
        t.q_stride = q_stride;
        t.out = static_cast<__nv_bfloat16*>(out);
        t.causal = causal;
        t.window = window;
        // a scale below zero turns the queries' sign, one of zero leaves no query
        t.scale_log2 = scale != 0.f ? fabsf(scale) * 1.4426950408889634f : 1.f;
        t.q_and = scale != 0.f ? 0xffffffffu : 0u;
        t.q_xor = scale < 0.f ? 0x80008000u : 0u;
        t.pieces = int(pieces);
        t.cluster = choose_cluster(p, pieces * p.hkv, cap);
        const cudaError_t e = p.d == 64 ? launch_tc<64>(t, p, page_maps(pool), s)
                                        : launch_tc<128>(t, p, page_maps(pool), s);
        return e == cudaSuccess ? PGD_OK : PGD_ERR_CUDA;
    }
    const AttendArgs a = {{cu_seqlens, block_table, seq_lens, B, total, max_blocks, p.block_size,
                           p.num_blocks, cap, p.err},
                          p.k, p.v, p.k_scale, p.v_scale, p.scale_per_block, Hq, p.hkv,
                          static_cast<const __nv_bfloat16*>(q), q_stride,
                          static_cast<__nv_bfloat16*>(out), causal, window,
                          scale * 1.4426950408889634f};
    const int64_t ctas = ((int64_t)total * Hq + kWarps - 1) / kWarps;
    if (ctas > INT32_MAX) return PGD_ERR_SHAPE;
    if (p.dtype == PGD_FP8_E4M3)
        attend_simple_kernel<PGD_FP8_E4M3, 128><<<(unsigned)ctas, kWarps * 32, 0, s>>>(a);
    else
        attend_simple_kernel<PGD_INT8, 128><<<(unsigned)ctas, kWarps * 32, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? PGD_OK : PGD_ERR_CUDA;
}
