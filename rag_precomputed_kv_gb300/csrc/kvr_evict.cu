// kvr_evict.cu -- a stitched cache cut to its heaviest rows.
//
// Per (request, layer, kv-head): of the n rows held, the first n_first, the
// last n_recent and the rows of largest weight between them stay, `keep` in
// all, in their order; equal weights go to the lowest row.  Row kept[i] moves
// to row i.  The stitched cache's rows sit at positions equal to their row
// (TurboRAG blog, "Position ID": contiguous positions), so a key that moves
// from row kept[i] to row i is turned by i - kept[i], the same re-rotation
// that stitched it (CoinRAG blog section 2.3); values and weights are copied.
//
// Two kernels.  k_evict_select finds each unit's kept rows: the threshold
// weight by a radix select over order-preserving integer keys, then the rows
// at or above it in order.  k_evict_move gathers the kept rows: a pure HBM
// stream like the stitch.
#include <cuda_bf16.h>

#include <algorithm>

#include "kvr_internal.cuh"

namespace kvr {

namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMoveThreads = 256;

// Integer key in the order of the weights: NaN lowest, then -inf .. +inf, both
// zeros alike.
__device__ __forceinline__ uint32_t weight_key(float w)
{
    if (w != w)
        return 0u;
    const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// 16-byte vectors of E elements of a row, rotation of a (lo, hi) pair of them.
template <typename T>
struct RowVec;

template <>
struct RowVec<__nv_bfloat16> {
    static constexpr int E = 8;
    __device__ static void rotate(uint4 &lo, uint4 &hi, const float *c, const float *s, bool il)
    {
        if (il)
            rotate_bf16x8_il(lo, hi, c, s);
        else
            rotate_bf16x8(lo, hi, c, s);
    }
};

template <>
struct RowVec<float> {
    static constexpr int E = 4;
    __device__ static void rotate(uint4 &lo, uint4 &hi, const float *c, const float *s, bool il)
    {
        float *x = reinterpret_cast<float *>(&lo);
        float *y = reinterpret_cast<float *>(&hi);
        if (il) {
            // pairs (x0, x1), (x2, x3) of lo with c[0], c[1]; of hi with c[2], c[3]
            float *v[2] = {x, y};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const float a0 = v[h][2 * p], a1 = v[h][2 * p + 1];
                    const float cc = c[2 * h + p], ss = s[2 * h + p];
                    v[h][2 * p] = fmaf(a0, cc, -a1 * ss);
                    v[h][2 * p + 1] = fmaf(a0, ss, a1 * cc);
                }
            }
            return;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float xo = fmaf(x[e], c[e], -y[e] * s[e]);
            const float yo = fmaf(x[e], s[e], y[e] * c[e]);
            x[e] = xo;
            y[e] = yo;
        }
    }
};

}  // namespace

// One CTA per (request, unit).  The threshold is found 8 bits at a time: a
// histogram of the candidates' next digit, and the digit in which the k-th
// largest falls.  Each warp then owns one consecutive stretch of rows, counts
// what it keeps, and writes its rows behind the warps before it.
__global__ void __launch_bounds__(kSelThreads)
    k_evict_select(const __grid_constant__ EvictArgs a, const __grid_constant__ EvictTable rt)
{
    const DevEvict *reqs = a.reqs ? a.reqs : rt.reqs;
    const int b = (int)(blockIdx.x / (unsigned)a.units), lh = (int)(blockIdx.x % (unsigned)a.units);
    const DevEvict rq = reqs[b];
    int32_t *kept = a.kept + rq.kept0 + (int64_t)lh * rq.keep;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (rq.keep == rq.n) {
        for (int i = threadIdx.x; i < rq.n; i += kSelThreads)
            kept[i] = i;
        return;
    }
    const float *w = a.weights + rq.src_row0 + (int64_t)lh * rq.src_cap;
    const int lo = a.n_first, hi = rq.n - a.n_recent;   // rows that compete
    const int k = rq.keep - a.n_first - a.n_recent;     // how many of them stay

    __shared__ int hist[256];
    __shared__ uint32_t s_digit;
    __shared__ int s_left;
    __shared__ int s_gt[kSelWarps], s_eq[kSelWarps];
    uint32_t prefix = 0;   // the threshold's leading digits
    int left = k;          // how many of the rows with those digits stay
    for (int shift = 24; shift >= 0 && k > 0; shift -= 8) {
        for (int i = threadIdx.x; i < 256; i += kSelThreads)
            hist[i] = 0;
        __syncthreads();
        for (int i = lo + (int)threadIdx.x; i < hi; i += kSelThreads) {
            const uint32_t key = weight_key(w[i]);
            if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8)))
                atomicAdd(&hist[(key >> shift) & 255], 1);
        }
        __syncthreads();
        if (warp == 0) {
            // lane l holds digits 255 - 8l .. 248 - 8l (descending)
            int c[8], sum = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                c[e] = hist[255 - 8 * lane - e];
                sum += c[e];
            }
            int incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o)
                    incl += v;
            }
            int above = incl - sum;   // rows of larger digits
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (above < left && left <= above + c[e]) {
                    s_digit = 255 - 8 * lane - e;
                    s_left = left - above;
                }
                above += c[e];
            }
        }
        __syncthreads();
        prefix |= s_digit << shift;
        left = s_left;
        __syncthreads();
    }
    // `left` rows with key == prefix stay, the lowest ones; all with key > prefix
    const int seg = (rq.n + kSelThreads - 1) / kSelThreads * 32;   // rows of a warp
    const int r0 = warp * seg, r1 = min(rq.n, r0 + seg);
    auto cls = [&](int i, bool &gt, bool &eq) {
        gt = eq = false;
        if (i >= r1)
            return;
        if (i < lo || i >= hi) {
            gt = true;
        } else if (k > 0) {
            const uint32_t key = weight_key(w[i]);
            gt = key > prefix;
            eq = key == prefix;
        }
    };
    int n_gt = 0, n_eq = 0;
    for (int i0 = r0; i0 < r1; i0 += 32) {
        bool gt, eq;
        cls(i0 + lane, gt, eq);
        n_gt += __popc(__ballot_sync(0xffffffffu, gt));
        n_eq += __popc(__ballot_sync(0xffffffffu, eq));
    }
    if (lane == 0) {
        s_gt[warp] = n_gt;
        s_eq[warp] = n_eq;
    }
    __syncthreads();
    int gt_before = 0, eq_before = 0;
    for (int x = 0; x < warp; ++x) {
        gt_before += s_gt[x];
        eq_before += s_eq[x];
    }
    const unsigned below = (1u << lane) - 1u;
    for (int i0 = r0; i0 < r1; i0 += 32) {
        bool gt, eq;
        cls(i0 + lane, gt, eq);
        const unsigned bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
        const int g = gt_before + __popc(bg & below), e = eq_before + __popc(be & below);
        if (gt || (eq && e < left))
            kept[g + min(e, left)] = i0 + lane;
        gt_before += __popc(bg);
        eq_before += __popc(be);
    }
}

// A piece is kEvictChunk kept rows of one unit.  TPR threads a row, thread j
// holding 16-byte vector j of each row half (so that both halves of a RoPE
// pair are in one thread).  To another block, every piece is a CTA.  In place,
// a CTA walks its unit's pieces in order: a piece's sources lie at or behind
// its own rows, so once the piece is read (barrier), writing it only
// overwrites rows that were read before.
template <typename T, int D>
__global__ void __launch_bounds__(kMoveThreads)
    k_evict_move(const __grid_constant__ EvictArgs a, const __grid_constant__ EvictTable rt)
{
    constexpr int E = RowVec<T>::E, H2 = D / 2, TPR = H2 / E, RPP = kMoveThreads / TPR;
    constexpr int NR = (kEvictChunk + RPP - 1) / RPP;   // rows of a thread
    const DevEvict *reqs = a.reqs ? a.reqs : rt.reqs;
    int b, lh, c_first, c_end;
    if (a.in_place) {
        b = (int)(blockIdx.x / (unsigned)a.units);
        lh = (int)(blockIdx.x % (unsigned)a.units);
        c_first = 0;
        c_end = max(1, (reqs[b].keep + kEvictChunk - 1) / kEvictChunk);
    } else {
        int lo = 0, hi = a.n_reqs - 1;
        while (lo < hi) {   // the last request whose first piece is <= blockIdx.x
            const int mid = (lo + hi + 1) >> 1;
            if (reqs[mid].chunk0 <= (int)blockIdx.x)
                lo = mid;
            else
                hi = mid - 1;
        }
        b = lo;
        const int n_c = max(1, (reqs[b].keep + kEvictChunk - 1) / kEvictChunk);
        const int local = (int)blockIdx.x - reqs[b].chunk0;
        lh = local / n_c;
        c_first = local - lh * n_c;
        c_end = c_first + 1;
    }
    const DevEvict rq = reqs[b];
    const int n_chunks = max(1, (rq.keep + kEvictChunk - 1) / kEvictChunk);
    const int32_t *kept = a.kept + rq.kept0 + (int64_t)lh * rq.keep;
    const int64_t src0 = rq.src_row0 + (int64_t)lh * rq.src_cap, dst0 = rq.dst_row0 + (int64_t)lh * rq.dst_cap;
    const T *sk = static_cast<const T *>(a.cache_k) + src0 * D, *sv = static_cast<const T *>(a.cache_v) + src0 * D;
    T *dk = static_cast<T *>(a.dst_k) + dst0 * D, *dv = static_cast<T *>(a.dst_v) + dst0 * D;
    const float *sw = a.weights + src0;
    float *dw = a.dst_weights ? a.dst_weights + dst0 : nullptr;
    const int j = threadIdx.x % TPR, rr = threadIdx.x / TPR;
    for (int c = c_first; c < c_end; ++c) {
        uint4 k[NR][2], v[NR][2];
        int src[NR];
        float wt = 0.f;
#pragma unroll
        for (int x = 0; x < NR; ++x) {
            const int i = c * kEvictChunk + x * RPP + rr;
            src[x] = -1;
            if (x * RPP + rr < kEvictChunk && i < rq.keep)
                src[x] = kept[i];
        }
#pragma unroll
        for (int x = 0; x < NR; ++x) {
            if (src[x] < 0)
                continue;
            const int64_t o = (int64_t)src[x] * D + j * E;
            k[x][0] = *reinterpret_cast<const uint4 *>(sk + o);
            k[x][1] = *reinterpret_cast<const uint4 *>(sk + o + H2);
            v[x][0] = *reinterpret_cast<const uint4 *>(sv + o);
            v[x][1] = *reinterpret_cast<const uint4 *>(sv + o + H2);
        }
        const int wi = c * kEvictChunk + (int)threadIdx.x;
        const bool has_w = dw && threadIdx.x < kEvictChunk && wi < rq.keep;
        if (has_w)
            wt = sw[kept[wi]];
        if (a.in_place)
            __syncthreads();
        if (has_w)
            dw[wi] = wt;
#pragma unroll
        for (int x = 0; x < NR; ++x) {
            if (src[x] < 0)
                continue;
            const int i = c * kEvictChunk + x * RPP + rr;
            const int delta = i - src[x];
            if (delta != 0 && !a.keep_rotation) {
                float cs[E], sn[E];
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float2 r = rope_cs(a.rope, H2, delta, rope_pair(a.interleaved, D, E, j, e));
                    cs[e] = r.x;
                    sn[e] = r.y;
                }
                RowVec<T>::rotate(k[x][0], k[x][1], cs, sn, a.interleaved);
            }
            const int64_t o = (int64_t)i * D + j * E;
            *reinterpret_cast<uint4 *>(dk + o) = k[x][0];
            *reinterpret_cast<uint4 *>(dk + o + H2) = k[x][1];
            *reinterpret_cast<uint4 *>(dv + o) = v[x][0];
            *reinterpret_cast<uint4 *>(dv + o + H2) = v[x][1];
        }
    }
    // the rows behind the kept ones start at no weight
    if (dw && c_end == n_chunks) {
        if (a.in_place)
            __syncthreads();
        for (int i = rq.keep + (int)threadIdx.x; i < rq.dst_cap; i += kMoveThreads)
            dw[i] = 0.f;
    }
}

cudaError_t launch_evict(const EvictArgs &a, const EvictTable &rt, int dtype, int head_dim, cudaStream_t s)
{
    const int64_t ctas = (int64_t)a.n_reqs * a.units;
    const int64_t move = a.in_place ? ctas : a.n_chunks;
    if (ctas > 0x7fffffff || move > 0x7fffffff)
        return cudaErrorInvalidValue;
    k_evict_select<<<(unsigned)ctas, kSelThreads, 0, s>>>(a, rt);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    if (dtype == KVR_DTYPE_BF16 && head_dim == 128)
        k_evict_move<__nv_bfloat16, 128><<<(unsigned)move, kMoveThreads, 0, s>>>(a, rt);
    else if (dtype == KVR_DTYPE_BF16 && head_dim == 64)
        k_evict_move<__nv_bfloat16, 64><<<(unsigned)move, kMoveThreads, 0, s>>>(a, rt);
    else if (dtype == KVR_DTYPE_FP32 && head_dim == 128)
        k_evict_move<float, 128><<<(unsigned)move, kMoveThreads, 0, s>>>(a, rt);
    else if (dtype == KVR_DTYPE_FP32 && head_dim == 64)
        k_evict_move<float, 64><<<(unsigned)move, kMoveThreads, 0, s>>>(a, rt);
    else
        return cudaErrorInvalidValue;
    return cudaGetLastError();
}

}  // namespace kvr
