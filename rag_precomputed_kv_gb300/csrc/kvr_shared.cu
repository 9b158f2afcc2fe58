// kvr_shared.cu -- query attention over a prefix shared by a group of
// requests, on the CUDA cores.
//
// Requests that were answered from the same retrieved spans have the same
// stitched prefix (CoinRAG blog section 2.3, C_ctx); it is stitched once, into
// a block of its own, and each request keeps only what follows it.  Query
// token t of request b sits at position p = P_g + S_b + t, its key and value
// were appended at own row S_b + t, and it attends to the P_g prefix rows and
// to own rows 0..S_b + t.
//
// The path for fp32 caches and head_dim 64.  One CTA per (layer,
// query token, query head), the keys split in as many stretches as it has warps; each lane holds
// head_dim / 32 elements; eight keys at a time, so that their loads and
// reductions over the warp overlap; online softmax in fp32, the warps' states
// added in warp order.  Three requests with 200 rows each: 11.4 us a call,
// all of it latency (four warps a row 18.6; one, four keys at a time, 47).
#include <cuda_bf16.h>

#include "kvr_internal.cuh"

namespace kvr {

namespace {

__device__ __forceinline__ float sh_to_f(float x) { return x; }
__device__ __forceinline__ float sh_to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T sh_from_f(float x);
template <>
__device__ __forceinline__ float sh_from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 sh_from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

}  // namespace

template <typename T, int D, int kShWarps>
__global__ void __launch_bounds__(32 * kShWarps)
    k_shared_simt(const __grid_constant__ SharedArgs a, const __grid_constant__ SharedTable rt)
{
    pdl_wait_prerequisites();
    const DevShared *reqs = a.reqs ? a.reqs : rt.reqs;
    constexpr int PL = D / 32, KU = 8;
    const int64_t w = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int Hq = a.n_q_heads;
    const int h = (int)(w % Hq);
    const int tok = (int)((w / Hq) % a.total_q);
    const int l = (int)(w / Hq / a.total_q);

    // the request of this token: the last one that starts at or before it
    int lo = 0, hi = a.n_reqs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (reqs[mid].q_off <= tok)
            lo = mid;
        else
            hi = mid - 1;
    }
    const DevShared rq = reqs[lo];
    const int t = tok - rq.q_off;
    const int pos = rq.pre_len + rq.own + t;
    const int kvh = h / (Hq / a.n_kv_heads);
    const int lh = l * a.n_kv_heads + kvh;

    const T *qp = static_cast<const T *>(a.q) + (((int64_t)l * a.total_q + tok) * Hq + h) * D;
    float qv[PL];
#pragma unroll
    for (int k = 0; k < PL; ++k)
        qv[k] = sh_to_f(qp[lane + 32 * k]);
    if (a.interleaved) {
        // pairs (x_2i, x_2i+1): element lane + 32k and its neighbour lane ^ 1
#pragma unroll
        for (int k = 0; k < PL; ++k) {
            const float2 cs = rope_cs(a.rope, D / 2, pos, (lane + 32 * k) >> 1);
            const float other = __shfl_xor_sync(0xffffffffu, qv[k], 1);
            qv[k] = (lane & 1) ? fmaf(other, cs.y, qv[k] * cs.x) : fmaf(qv[k], cs.x, -other * cs.y);
        }
    } else {
#pragma unroll
        for (int k = 0; k < PL / 2; ++k) {
            const float2 cs = rope_cs(a.rope, D / 2, pos, lane + 32 * k);
            const float x = qv[k], y = qv[k + PL / 2];
            qv[k] = fmaf(x, cs.x, -y * cs.y);
            qv[k + PL / 2] = fmaf(x, cs.y, y * cs.x);
        }
    }

    float m = -INFINITY, lsum = 0.f, acc[PL];
#pragma unroll
    for (int k = 0; k < PL; ++k)
        acc[k] = 0.f;
    // rows j_lo..j_hi-1 of a block (none: an empty stretch)
    auto attend = [&](const T *kp, const T *vp, int j_lo, int j_hi) {
        for (int j0 = j_lo; j0 < j_hi; j0 += KU) {
            float d[KU], v[KU][PL];
#pragma unroll
            for (int u = 0; u < KU; ++u) {
                d[u] = 0.f;
                const int64_t row = min(j0 + u, j_hi - 1);
#pragma unroll
                for (int k = 0; k < PL; ++k) {
                    d[u] = fmaf(qv[k], sh_to_f(kp[row * D + lane + 32 * k]), d[u]);
                    v[u][k] = sh_to_f(vp[row * D + lane + 32 * k]);
                }
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
#pragma unroll
                for (int u = 0; u < KU; ++u)
                    d[u] += __shfl_xor_sync(0xffffffffu, d[u], off);
            float mn = m;
#pragma unroll
            for (int u = 0; u < KU; ++u) {
                d[u] = j0 + u < j_hi ? d[u] * a.scale_log2 : -INFINITY;
                mn = fmaxf(mn, d[u]);
            }
            // (mn stays -inf only while every score so far is -inf or NaN)
            const float ref = mn == -INFINITY ? 0.f : mn;
            const float corr = exp2f(m - ref);
            lsum *= corr;
#pragma unroll
            for (int k = 0; k < PL; ++k)
                acc[k] *= corr;
#pragma unroll
            for (int u = 0; u < KU; ++u) {
                if (j0 + u >= j_hi)
                    break;
                const float p = exp2f(d[u] - ref);
                lsum += p;
#pragma unroll
                for (int k = 0; k < PL; ++k)
                    acc[k] = fmaf(p, v[u][k], acc[k]);
            }
            m = mn;
        }
    };
    // warp x: the x-th stretch of the prefix rows and of the own rows
    const int64_t pre = (rq.pre_row0 + (int64_t)lh * rq.pre_cap) * D, own = (rq.cache_row0 + (int64_t)lh * rq.cap) * D;
    const int n_own = rq.own + t + 1;
    if (rq.pre_len > 0)
        attend(static_cast<const T *>(a.prefix_k) + pre, static_cast<const T *>(a.prefix_v) + pre,
               (int)((int64_t)rq.pre_len * warp / kShWarps), (int)((int64_t)rq.pre_len * (warp + 1) / kShWarps));
    attend(static_cast<const T *>(a.cache_k) + own, static_cast<const T *>(a.cache_v) + own, (int)((int64_t)n_own * warp / kShWarps),
           (int)((int64_t)n_own * (warp + 1) / kShWarps));
    __shared__ float s_m[kShWarps], s_l[kShWarps], s_acc[kShWarps][D];
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = lsum;
    }
#pragma unroll
    for (int k = 0; k < PL; ++k)
        s_acc[warp][lane + 32 * k] = acc[k];
    __syncthreads();
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int x = 0; x < kShWarps; ++x)
        M = fmaxf(M, s_l[x] == 0.f ? -INFINITY : s_m[x]);   // (a sum of 0: no key counts)
    float wx[kShWarps];
#pragma unroll
    for (int x = 0; x < kShWarps; ++x) {
        wx[x] = s_l[x] == 0.f ? 0.f : exp2f(s_m[x] - M);
        L += s_l[x] * wx[x];
    }
    if (threadIdx.x == 0 && !(L > 0.f && L < INFINITY))
        atomicCAS(a.err, kDevOk, kDevBadInput);
    const float inv = 1.f / L;
    T *op = static_cast<T *>(a.out) + (((int64_t)l * a.total_q + tok) * Hq + h) * D;
    if ((int)threadIdx.x < D) {
        float o = 0.f;
#pragma unroll
        for (int x = 0; x < kShWarps; ++x)
            o = fmaf(s_acc[x][threadIdx.x], wx[x], o);
        op[threadIdx.x] = sh_from_f<T>(o * inv);
    }
}

template <int kShWarps>
static cudaError_t launch_w(const SharedArgs &a, const SharedTable &rt, int dtype, int head_dim, int64_t blocks, cudaStream_t s)
{
    using Kernel = void (*)(const SharedArgs, const SharedTable);
    const Kernel k = head_dim == 128 ? (dtype == KVR_DTYPE_BF16 ? k_shared_simt<__nv_bfloat16, 128, kShWarps> : k_shared_simt<float, 128, kShWarps>)
                     : head_dim == 64 ? (dtype == KVR_DTYPE_BF16 ? k_shared_simt<__nv_bfloat16, 64, kShWarps> : k_shared_simt<float, 64, kShWarps>)
                                      : nullptr;
    return k ? launch_pdl(k, blocks, 32 * kShWarps, 0, true, s, a, rt) : cudaErrorInvalidValue;
}

cudaError_t launch_shared_simt(const SharedArgs &a, const SharedTable &rt, int dtype, int head_dim, int n_sms, cudaStream_t s)
{
    // Sixteen warps a row where rows are few, four where they fill the SMs: 32 rows
    // of 2,000 keys 37 us a call against 123; 1,280 rows of 750 keys 74 against 62.
    const int64_t blocks = (int64_t)a.n_layers * a.total_q * a.n_q_heads;
    return blocks <= 2 * (int64_t)n_sms ? launch_w<16>(a, rt, dtype, head_dim, blocks, s)
                                        : launch_w<4>(a, rt, dtype, head_dim, blocks, s);
}

}  // namespace kvr
