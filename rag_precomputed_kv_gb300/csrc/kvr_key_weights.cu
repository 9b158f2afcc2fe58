// kvr_key_weights.cu -- attention weight per cached key, on the CUDA cores.
//
// For every (request, layer, kv-head) and key row j < P_b + Lq_b:
//     w[j] (+)= sum over query tokens t and the G query heads g of the kv head
//               of softmax_j(scale * <rot(q_tg, P_b + t), k_j>),  j <= P_b + t,
// the probabilities of the query attention (CoinRAG blog section 2.3,
// KV_M(q; C_ctx)) summed over the queries: what each cached row was read for.
//
// The path for fp32 caches and head_dim 64.  One CTA per (request, unit); 16
// query rows at a time, rotated into shared memory; a thread owns the keys
// j = tid + 256 i and computes a key's 16 scores from one read of its row.
// Two passes over the keys: the rows' maxima and sums, then the weights, so
// nothing of the size (rows x keys) is stored, and every weight is summed by
// one thread in row order.
//
// Bound by latency at the sizes it is for: 16 tokens x 2 heads on 219 keys, two
// units: 26.7 us a call, two CTAs of two passes over three row blocks.
#include <cuda_bf16.h>

#include "kvr_internal.cuh"

namespace kvr {

namespace {

constexpr int kWThreads = 256;
constexpr int kWRows = 16;

template <typename T>
__device__ __forceinline__ void unpack16(const uint4 &u, float *f);
template <>
__device__ __forceinline__ void unpack16<float>(const uint4 &u, float *f)
{
    f[0] = __uint_as_float(u.x);
    f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z);
    f[3] = __uint_as_float(u.w);
}
template <>
__device__ __forceinline__ void unpack16<__nv_bfloat16>(const uint4 &u, float *f)
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ float w_to_f(float x) { return x; }
__device__ __forceinline__ float w_to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

}  // namespace

template <typename T, int D>
__global__ void __launch_bounds__(kWThreads)
    k_key_weights_simt(const __grid_constant__ WeightsArgs a, const __grid_constant__ ReqTable rt)
{
    constexpr int E = 16 / (int)sizeof(T), H2 = D / 2;
    const DevReq *reqs = a.reqs ? a.reqs : rt.reqs;
    const int units = a.n_layers * a.n_kv_heads;
    const DevReq rq = reqs[blockIdx.x / (unsigned)units];
    const int lh = (int)(blockIdx.x % (unsigned)units);
    const int l = lh / a.n_kv_heads, h = lh - l * a.n_kv_heads;
    const int G = a.n_q_heads / a.n_kv_heads;
    const int m_rows = rq.q_len * G, n = rq.prefix + rq.q_len;
    const int64_t blk = rq.cache_row0 + (int64_t)lh * rq.cap;
    const T *kp = static_cast<const T *>(a.cache_k) + blk * D;
    float *w = a.weights + blk;

    __shared__ __align__(16) float sq[kWRows][D];
    __shared__ float red_m[kWThreads / 32][kWRows], red_l[kWThreads / 32][kWRows], fin_m[kWRows], fin_i[kWRows];

    if (m_rows == 0) {   // a sum over no queries
        if (!a.accumulate)
            for (int j = threadIdx.x; j < n; j += kWThreads)
                w[j] = 0.f;
        return;
    }
    for (int r0 = 0; r0 < m_rows; r0 += kWRows) {
        const int nr = min(kWRows, m_rows - r0);
        // the batch's query rows, rotated, times the scale (log2 units)
        for (int x = threadIdx.x; x < kWRows * H2; x += kWThreads) {
            const int r = x / H2, i = x - r * H2;
            float x0 = 0.f, x1 = 0.f;
            const int d0 = a.interleaved ? 2 * i : i, d1 = a.interleaved ? 2 * i + 1 : i + H2;
            if (r < nr) {
                const int t = (r0 + r) / G, g = (r0 + r) - t * G;
                const T *q = static_cast<const T *>(a.q) +
                             (((int64_t)l * a.total_q + rq.q_off + t) * a.n_q_heads + h * G + g) * D;
                const float2 cs = rope_cs(a.rope, H2, rq.prefix + t, i);
                const float u = w_to_f(q[d0]), v = w_to_f(q[d1]);
                x0 = fmaf(u, cs.x, -v * cs.y);
                x1 = fmaf(u, cs.y, v * cs.x);
            }
            sq[r][d0] = x0;
            sq[r][d1] = x1;
        }
        __syncthreads();
        auto scores = [&](int j, float *s) {
#pragma unroll
            for (int r = 0; r < kWRows; ++r)
                s[r] = 0.f;
#pragma unroll 8
            for (int d = 0; d < D; d += E) {
                float f[E];
                unpack16<T>(*reinterpret_cast<const uint4 *>(kp + (int64_t)j * D + d), f);
#pragma unroll
                for (int r = 0; r < kWRows; ++r)
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        s[r] = fmaf(sq[r][d + e], f[e], s[r]);
            }
            // rows that do not see the key: their token lies before it
            const int r_min = (j - rq.prefix) * G - r0;
#pragma unroll
            for (int r = 0; r < kWRows; ++r)
                s[r] = (r >= r_min && r < nr) ? s[r] * a.scale_log2 : -INFINITY;
        };
        // a cache of at most one key a thread keeps its scores between the passes
        const bool one = n <= kWThreads;
        float s[kWRows], m[kWRows], ls[kWRows];
#pragma unroll
        for (int r = 0; r < kWRows; ++r) {
            m[r] = -INFINITY;
            ls[r] = 0.f;
        }
        for (int j = threadIdx.x; j < n; j += kWThreads) {
            scores(j, s);
#pragma unroll
            for (int r = 0; r < kWRows; ++r) {
                if (s[r] != -INFINITY) {   // (NaN scores go through)
                    const float mn = fmaxf(m[r], s[r]);
                    ls[r] = ls[r] * exp2f(m[r] - mn) + exp2f(s[r] - mn);
                    m[r] = mn;
                }
            }
        }
#pragma unroll
        for (int r = 0; r < kWRows; ++r) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const float mo = __shfl_xor_sync(0xffffffffu, m[r], o), lo = __shfl_xor_sync(0xffffffffu, ls[r], o);
                const float mn = fmaxf(m[r], mo);
                const float c0 = mn == -INFINITY ? 1.f : exp2f(m[r] - mn), c1 = mn == -INFINITY ? 1.f : exp2f(mo - mn);
                ls[r] = ls[r] * c0 + lo * c1;
                m[r] = mn;
            }
            if ((threadIdx.x & 31) == 0) {
                red_m[threadIdx.x >> 5][r] = m[r];
                red_l[threadIdx.x >> 5][r] = ls[r];
            }
        }
        __syncthreads();
        if (threadIdx.x < kWRows) {
            const int r = threadIdx.x;
            float mm = -INFINITY, ll = 0.f;
            for (int x = 0; x < kWThreads / 32; ++x)
                mm = fmaxf(mm, red_m[x][r]);
            for (int x = 0; x < kWThreads / 32; ++x)
                if (red_l[x][r] != 0.f)
                    ll += red_l[x][r] * (red_m[x][r] == -INFINITY ? 1.f : exp2f(red_m[x][r] - mm));
            fin_m[r] = mm == -INFINITY ? 0.f : mm;
            fin_i[r] = 1.f / ll;
            if (r < nr && !(ll > 0.f && ll < INFINITY))
                atomicCAS(a.err, kDevOk, kDevBadInput);
        }
        __syncthreads();
        for (int j = threadIdx.x; j < n; j += kWThreads) {
            float sum = 0.f;
            if (!one)
                scores(j, s);
#pragma unroll
            for (int r = 0; r < kWRows; ++r)
                if (s[r] != -INFINITY)
                    sum = fmaf(exp2f(s[r] - fin_m[r]), fin_i[r], sum);
            w[j] = (r0 > 0 || a.accumulate ? w[j] : 0.f) + sum;
        }
        __syncthreads();   // the batch's queries and statistics are read
    }
}

cudaError_t launch_weights_simt(const WeightsArgs &a, const ReqTable &rt, int dtype, int head_dim, cudaStream_t s)
{
    const int64_t ctas = (int64_t)a.n_reqs * a.n_layers * a.n_kv_heads;
    if (ctas > 0x7fffffff)
        return cudaErrorInvalidValue;
    if (dtype == KVR_DTYPE_BF16 && head_dim == 128)
        k_key_weights_simt<__nv_bfloat16, 128><<<(unsigned)ctas, kWThreads, 0, s>>>(a, rt);
    else if (dtype == KVR_DTYPE_BF16 && head_dim == 64)
        k_key_weights_simt<__nv_bfloat16, 64><<<(unsigned)ctas, kWThreads, 0, s>>>(a, rt);
    else if (dtype == KVR_DTYPE_FP32 && head_dim == 128)
        k_key_weights_simt<float, 128><<<(unsigned)ctas, kWThreads, 0, s>>>(a, rt);
    else if (dtype == KVR_DTYPE_FP32 && head_dim == 64)
        k_key_weights_simt<float, 64><<<(unsigned)ctas, kWThreads, 0, s>>>(a, rt);
    else
        return cudaErrorInvalidValue;
    return cudaGetLastError();
}

}  // namespace kvr
