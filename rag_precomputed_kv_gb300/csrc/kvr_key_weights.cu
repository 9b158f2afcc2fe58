// kvr_key_weights.cu -- attention weight per cached key, on the CUDA cores.
//
// For every (request, layer, kv-head) and key row j < P_b + Lq_b:
//     w[j] (+)= sum over query tokens t and the G query heads g of the kv head
//               of softmax_j(scale * <rot(q_tg, P_b + t), k_j>),  j <= P_b + t,
// the probabilities of the query attention (CoinRAG blog section 2.3,
// KV_M(q; C_ctx)) summed over the queries: what each cached row was read for.
//
// The path for fp32 caches and head_dim 64.  A cluster of up to eight CTAs per
// (request, unit) splits its keys; 32 query rows at a time, rotated into shared
// memory; a thread owns a key and eight of the rows (with fewer rows there are
// more keys at a time), and computes their scores from one read of the key's row.
// Two passes over the keys: the rows' maxima and sums, which the CTAs exchange
// through distributed shared memory, then the weights, so nothing of the size
// (rows x keys) is stored; the threads of a key add their parts in row order.
//
// Bound by latency at the sizes it is for: 16 tokens x 2 heads on 219 keys, two
// units: 12.8 us a call; one token on 1,900 keys, six units: 14.2 us.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "kvr_tc_common.cuh"

namespace kvr {

namespace {

constexpr int kWThreads = 1024;
constexpr int kWPer = 8;              // rows of a thread
constexpr int kWRows = 4 * kWPer;     // rows at a time, by at most four threads of a key
constexpr int kWMaxCluster = 8;
__host__ __device__ constexpr int w_groups(int rows) { return rows > 2 * kWPer ? 4 : rows > kWPer ? 2 : 1; }

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
    k_key_weights_simt(const __grid_constant__ WeightsArgs a, const __grid_constant__ ReqTable rt, const int n_cluster)
{
    constexpr int E = 16 / (int)sizeof(T), H2 = D / 2;
    pdl_wait_prerequisites();
    const DevReq *reqs = a.reqs ? a.reqs : rt.reqs;
    const int units = a.n_layers * a.n_kv_heads;
    const int rank = (int)(blockIdx.x % (unsigned)n_cluster), unit_i = (int)(blockIdx.x / (unsigned)n_cluster);
    const DevReq rq = reqs[unit_i / units];
    const int lh = unit_i % units;
    const int l = lh / a.n_kv_heads, h = lh - l * a.n_kv_heads;
    const int G = a.n_q_heads / a.n_kv_heads;
    const int m_rows = rq.q_len * G, n = rq.prefix + rq.q_len;
    const int j_lo = (int)((int64_t)n * rank / n_cluster), j_hi = (int)((int64_t)n * (rank + 1) / n_cluster);
    const int64_t blk = rq.cache_row0 + (int64_t)lh * rq.cap;
    const T *kp = static_cast<const T *>(a.cache_k) + blk * D;
    float *w = a.weights + blk;

    __shared__ __align__(16) float sq[kWRows][D];
    __shared__ float red_m[kWThreads / 32][kWPer], red_l[kWThreads / 32][kWPer], fin_m[kWRows], fin_i[kWRows];
    __shared__ float part[kWThreads];
    __shared__ float2 peers[2][kWMaxCluster][kWRows];   // (max, sum) of the cluster's CTAs, by turns

    if (m_rows == 0) {   // a sum over no queries
        if (!a.accumulate)
            for (int j = j_lo + threadIdx.x; j < j_hi; j += kWThreads)
                w[j] = 0.f;
        return;
    }
    if (n_cluster > 1)
        tc::cluster_sync();   // (the CTAs of a cluster have started: their shared memory may be written)
    int turn = 0;
    for (int r0 = 0; r0 < m_rows; r0 += kWRows, turn ^= 1) {
        const int nr = min(kWRows, m_rows - r0), ng = w_groups(nr), keys = kWThreads / ng;
        const int lane_key = threadIdx.x % keys, row0 = threadIdx.x / keys * kWPer;
        // the batch's query rows, rotated
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
            for (int r = 0; r < kWPer; ++r)
                s[r] = 0.f;
#pragma unroll(16 / E)   // (more spill)
            for (int d = 0; d < D; d += E) {
                float f[E];
                unpack16<T>(*reinterpret_cast<const uint4 *>(kp + (int64_t)j * D + d), f);
#pragma unroll
                for (int r = 0; r < kWPer; ++r)
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        s[r] = fmaf(sq[row0 + r][d + e], f[e], s[r]);
            }
            // rows that do not see the key: their token lies before it
            const int r_min = max(j - rq.prefix, 0) * G - r0;   // (a far prefix times G passes 32 bits)
#pragma unroll
            for (int r = 0; r < kWPer; ++r)
                s[r] = (row0 + r >= r_min && row0 + r < nr) ? s[r] * a.scale_log2 : -INFINITY;
        };
        // at most one key a thread: its scores are kept between the passes
        const bool one = j_hi - j_lo <= keys;
        float s[kWPer], m[kWPer], ls[kWPer];
#pragma unroll
        for (int r = 0; r < kWPer; ++r) {
            m[r] = -INFINITY;
            ls[r] = 0.f;
        }
        for (int j = j_lo + lane_key; j < j_hi; j += keys) {
            scores(j, s);
#pragma unroll
            for (int r = 0; r < kWPer; ++r) {
                if (s[r] != -INFINITY) {   // (NaN scores go through)
                    const float mn = fmaxf(m[r], s[r]);
                    ls[r] = ls[r] * exp2f(m[r] - mn) + exp2f(s[r] - mn);
                    m[r] = mn;
                }
            }
        }
#pragma unroll
        for (int r = 0; r < kWPer; ++r) {
            float mw = m[r];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                mw = fmaxf(mw, __shfl_xor_sync(0xffffffffu, mw, o));
            if (ls[r] != 0.f)   // (NaN sums go through)
                ls[r] *= mw == -INFINITY ? 1.f : exp2f(m[r] - mw);
            m[r] = mw;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                ls[r] += __shfl_xor_sync(0xffffffffu, ls[r], o);
            if ((threadIdx.x & 31) == 0) {
                red_m[threadIdx.x >> 5][r] = m[r];
                red_l[threadIdx.x >> 5][r] = ls[r];
            }
        }
        __syncthreads();
        // (max, sum) pairs added in order
        auto join = [](float2 &x, float2 v) {
            if (v.y == 0.f)   // no key
                return;
            const float mn = fmaxf(x.x, v.x);
            x.y = (x.y == 0.f ? 0.f : x.y * (mn == -INFINITY ? 1.f : exp2f(x.x - mn))) +
                  v.y * (mn == -INFINITY ? 1.f : exp2f(v.x - mn));
            x.x = mn;
        };
        const int row = threadIdx.x;
        float2 st = make_float2(-INFINITY, 0.f);
        if (row < ng * kWPer) {
            const int n_w = keys / 32, w0 = row / kWPer * n_w;
            for (int x = w0; x < w0 + n_w; ++x)
                join(st, make_float2(red_m[x][row % kWPer], red_l[x][row % kWPer]));
        }
        if (n_cluster > 1) {
            if (row < kWRows)
                for (int x = 0; x < n_cluster; ++x) {
                    const uint32_t dst = tc::mapa_rank(tc::smem_u32(&peers[turn][rank][row]), (uint32_t)x);
                    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(dst), "f"(st.x), "f"(st.y) : "memory");
                }
            // (by the time a CTA writes a turn's places again, all have passed the
            // other turn's barrier, behind their reads of this one's)
            tc::cluster_sync();
            st = make_float2(-INFINITY, 0.f);
            if (row < kWRows)
                for (int x = 0; x < n_cluster; ++x)
                    join(st, peers[turn][x][row]);
        }
        if (row < kWRows) {
            fin_m[row] = st.x == -INFINITY ? 0.f : st.x;
            fin_i[row] = 1.f / st.y;
            if (row < nr && rank == 0 && !(st.y > 0.f && st.y < INFINITY))
                atomicCAS(a.err, kDevOk, kDevBadInput);
        }
        __syncthreads();
        for (int j0 = j_lo; j0 < j_hi; j0 += keys) {
            const int j = j0 + lane_key;
            float sum = 0.f;
            if (j < j_hi) {
                if (!one)
                    scores(j, s);
#pragma unroll
                for (int r = 0; r < kWPer; ++r)
                    if (s[r] != -INFINITY)
                        sum = fmaf(exp2f(s[r] - fin_m[row0 + r]), fin_i[row0 + r], sum);
            }
            part[threadIdx.x] = sum;
            __syncthreads();
            if (row0 == 0 && j < j_hi) {
                float all = part[lane_key];
                for (int g = 1; g < ng; ++g)
                    all += part[g * keys + lane_key];
                w[j] = (r0 > 0 || a.accumulate ? w[j] : 0.f) + all;
            }
            __syncthreads();
        }
    }
}

cudaError_t launch_weights_simt(const WeightsArgs &a, const ReqTable &rt, int dtype, int head_dim, int n_sms, cudaStream_t s)
{
    using Kernel = void (*)(const WeightsArgs, const ReqTable, const int);
    const Kernel k = head_dim == 128 ? (dtype == KVR_DTYPE_BF16 ? k_key_weights_simt<__nv_bfloat16, 128> : k_key_weights_simt<float, 128>)
                     : head_dim == 64 ? (dtype == KVR_DTYPE_BF16 ? k_key_weights_simt<__nv_bfloat16, 64> : k_key_weights_simt<float, 64>)
                                      : nullptr;
    if (!k)
        return cudaErrorInvalidValue;
    const int64_t units = (int64_t)a.n_reqs * a.n_layers * a.n_kv_heads;
    const int keys = kWThreads / w_groups((int)std::min<int64_t>(kWRows, (int64_t)a.max_q_len * (a.n_q_heads / a.n_kv_heads)));
    // keys of a unit to more CTAs while SMs are idle and a quarter of the threads
    // have one (until each has one: 18.4 and 23.1 us where it is 12.8 and 14.2)
    int c = 1;
    while (c < kWMaxCluster && units * c * 2 <= n_sms && a.max_rows > c * keys / 4)
        c *= 2;
    return launch_cluster(k, units * c, kWThreads, 0, c, s, a, rt, c);
}

}  // namespace kvr
