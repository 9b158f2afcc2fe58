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
// The path for fp32 caches and head_dim 64.  One warp per (layer, query token,
// query head); each lane holds head_dim / 32 elements; four keys at a time, so
// that their reductions over the warp overlap; online softmax in fp32.
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

template <typename T, int D>
__global__ void __launch_bounds__(128)
    k_shared_simt(const __grid_constant__ SharedArgs a, const __grid_constant__ SharedTable rt)
{
    const DevShared *reqs = a.reqs ? a.reqs : rt.reqs;
    constexpr int PL = D / 32, KU = 4;
    const int64_t w = (int64_t)blockIdx.x * 4 + threadIdx.x / 32;
    const int lane = threadIdx.x & 31;
    const int Hq = a.n_q_heads;
    if (w >= (int64_t)a.n_layers * a.total_q * Hq)
        return;
    const int h = (int)(w % Hq);
    const int tok = (int)((w / Hq) % a.total_q);
    const int l = (int)(w / Hq / a.total_q);

    // the request of this token: the last one that starts at or before it and has tokens
    int lo = 0, hi = a.n_reqs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (reqs[mid].q_off <= tok)
            lo = mid;
        else
            hi = mid - 1;
    }
    while (lo > 0 && reqs[lo].q_len == 0)
        --lo;
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
    // rows 0..n_vis-1 of a block (n_vis may be 0: an empty prefix)
    auto attend = [&](const T *kp, const T *vp, int n_vis) {
        for (int j0 = 0; j0 < n_vis; j0 += KU) {
            float d[KU];
#pragma unroll
            for (int u = 0; u < KU; ++u) {
                d[u] = 0.f;
                const int64_t row = min(j0 + u, n_vis - 1);
#pragma unroll
                for (int k = 0; k < PL; ++k)
                    d[u] = fmaf(qv[k], sh_to_f(kp[row * D + lane + 32 * k]), d[u]);
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
#pragma unroll
                for (int u = 0; u < KU; ++u)
                    d[u] += __shfl_xor_sync(0xffffffffu, d[u], off);
            float mn = m;
#pragma unroll
            for (int u = 0; u < KU; ++u) {
                d[u] = j0 + u < n_vis ? d[u] * a.scale_log2 : -INFINITY;
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
                if (j0 + u >= n_vis)
                    break;
                const float p = exp2f(d[u] - ref);
                lsum += p;
#pragma unroll
                for (int k = 0; k < PL; ++k)
                    acc[k] = fmaf(p, sh_to_f(vp[(int64_t)(j0 + u) * D + lane + 32 * k]), acc[k]);
            }
            m = mn;
        }
    };
    const int64_t pre = (rq.pre_row0 + (int64_t)lh * rq.pre_cap) * D, own = (rq.cache_row0 + (int64_t)lh * rq.cap) * D;
    if (rq.pre_len > 0)
        attend(static_cast<const T *>(a.prefix_k) + pre, static_cast<const T *>(a.prefix_v) + pre, rq.pre_len);
    attend(static_cast<const T *>(a.cache_k) + own, static_cast<const T *>(a.cache_v) + own, rq.own + t + 1);
    if (lane == 0 && !(lsum > 0.f && lsum < INFINITY))
        atomicCAS(a.err, kDevOk, kDevBadInput);
    T *op = static_cast<T *>(a.out) + (((int64_t)l * a.total_q + tok) * Hq + h) * D;
    const float inv = 1.f / lsum;
#pragma unroll
    for (int k = 0; k < PL; ++k)
        op[lane + 32 * k] = sh_from_f<T>(acc[k] * inv);
}

cudaError_t launch_shared_simt(const SharedArgs &a, const SharedTable &rt, int dtype, int head_dim, cudaStream_t s)
{
    const int64_t blocks = ((int64_t)a.n_layers * a.total_q * a.n_q_heads + 3) / 4;
    if (blocks == 0)
        return cudaSuccess;
    if (blocks > 0x7fffffff)
        return cudaErrorInvalidValue;
    if (dtype == KVR_DTYPE_BF16 && head_dim == 128)
        k_shared_simt<__nv_bfloat16, 128><<<(unsigned)blocks, 128, 0, s>>>(a, rt);
    else if (dtype == KVR_DTYPE_BF16 && head_dim == 64)
        k_shared_simt<__nv_bfloat16, 64><<<(unsigned)blocks, 128, 0, s>>>(a, rt);
    else if (dtype == KVR_DTYPE_FP32 && head_dim == 128)
        k_shared_simt<float, 128><<<(unsigned)blocks, 128, 0, s>>>(a, rt);
    else if (dtype == KVR_DTYPE_FP32 && head_dim == 64)
        k_shared_simt<float, 64><<<(unsigned)blocks, 128, 0, s>>>(a, rt);
    else
        return cudaErrorInvalidValue;
    return cudaGetLastError();
}

}  // namespace kvr
