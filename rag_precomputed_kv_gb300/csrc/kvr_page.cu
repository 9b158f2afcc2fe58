// kvr_page.cu -- the paged cache: rotation and append, packing to 4 bits and
// back, and attention on the CUDA cores.
//
// A cache that grows token by token, or shrinks to a window, lives in pages:
// row r of a request is row r % R of its page r / R, in any order in memory.
// Rows are a query's positions: a token appended at row r has its key turned by
// r (TurboRAG blog, "Position ID": contiguous positions).
#include <cuda_bf16.h>

#include <algorithm>

#include "kvr_page_common.cuh"

namespace kvr {

namespace {

using namespace page;

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
constexpr int kApThreads = 128;

template <typename T>
struct Vec;   // 16 bytes of a row in fp32
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void get(const uint4 &u, float *f)
    {
        f[0] = __uint_as_float(u.x);
        f[1] = __uint_as_float(u.y);
        f[2] = __uint_as_float(u.z);
        f[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 put(const float *f)
    {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void get(const uint4 &u, float *f)
    {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 put(const float *f)
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// x, y: 16-byte vectors of a row's two halves; (c, s) per pair, ordered as
// rope_pair says.
template <typename T>
__device__ __forceinline__ void rotate_halves(uint4 &x, uint4 &y, const float2 *cs, bool il)
{
    constexpr int N = Vec<T>::N;
    float a[N], b[N];
    Vec<T>::get(x, a);
    Vec<T>::get(y, b);
    if (!il) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float u = a[e], w = b[e];
            a[e] = fmaf(u, cs[e].x, -(w * cs[e].y));
            b[e] = fmaf(u, cs[e].y, w * cs[e].x);
        }
    } else {
#pragma unroll
        for (int e = 0; e < N / 2; ++e) {
            float u = a[2 * e], w = a[2 * e + 1];
            a[2 * e] = fmaf(u, cs[e].x, -(w * cs[e].y));
            a[2 * e + 1] = fmaf(u, cs[e].y, w * cs[e].x);
            u = b[2 * e], w = b[2 * e + 1];
            b[2 * e] = fmaf(u, cs[N / 2 + e].x, -(w * cs[N / 2 + e].y));
            b[2 * e + 1] = fmaf(u, cs[N / 2 + e].y, w * cs[N / 2 + e].x);
        }
    }
    x = Vec<T>::put(a);
    y = Vec<T>::put(b);
}

}  // namespace

// A group of D / 2 / N threads per token: each holds a 16-byte vector of both
// halves of a row, its (cos, sin) once for all the units that its CTA takes.  Bound by
// HBM: 2,592 rows, 112 units, 47 us = 6.3 TB/s read and written, 0.94 of the copy rate (50 us
// turned).  A serving batch's 64 rows, 288 units (19 MB): 7.1 us in a replayed graph of calls on
// eight caches, 2.8 at the copy rate, of which a thread's chain (its request by bisection, a page
// number, the rotation, a row) is the larger part; a call by itself takes the host 10 to 13 us.
template <typename T, int D>
__global__ void __launch_bounds__(kApThreads)
    k_page_append(const __grid_constant__ PageArgs a, const __grid_constant__ PageTable t)
{
    constexpr int N = Vec<T>::N, kPer = D / 2 / N, kTokens = kApThreads / kPer;
    pdl_wait_prerequisites();   // (uploaded tables too are read behind it)
    pdl_launch_dependents();
    const DevPageReq *reqs = a.reqs ? a.reqs : t.reqs;
    const int32_t *ids = a.reqs ? a.ids : t.ids;
    const int units = a.n_layers * a.n_kv_heads, unit_blocks = (units + a.per_cta - 1) / a.per_cta;
    const int64_t tb = blockIdx.x / (unsigned)unit_blocks;
    const int u0 = (int)(blockIdx.x % (unsigned)unit_blocks) * a.per_cta, u1 = min(units, u0 + a.per_cta);
    const int j = threadIdx.x % kPer;
    const int64_t tok = tb * kTokens + threadIdx.x / kPer;
    if (tok >= a.total_q)
        return;
    const DevPageReq &rq = reqs[request_of(reqs, a.n_reqs, (int)tok)];
    const int row = rq.pos0 + (int)(tok - rq.q_off), pg = page_of(a, row);
    const int64_t dst0 = (int64_t)page_id(rq, ids, pg) * a.g.s_page + (int64_t)(row - pg * a.g.rows) * D + N * j;
    float2 cs[N];
    const bool il = a.interleaved != 0;
    if (!a.turned)
#pragma unroll
        for (int e = 0; e < N; ++e)
            cs[e] = rope_cs(a.rope, D / 2, row, rope_pair(il, D, N, j, e));
    const T *k = static_cast<const T *>(a.k) + tok * a.s_tok + N * j, *v = static_cast<const T *>(a.v) + tok * a.s_tok + N * j;
    T *pk = static_cast<T *>(a.g.k) + dst0, *pv = static_cast<T *>(a.g.v) + dst0;
#pragma unroll 2
    for (int u = u0; u < u1; ++u) {
        const int l = u / a.n_kv_heads, h = u - l * a.n_kv_heads;
        const int64_t src = l * a.s_layer + h * a.s_head, dst = l * a.g.s_layer + h * a.g.s_head;
        uint4 x = *reinterpret_cast<const uint4 *>(k + src), y = *reinterpret_cast<const uint4 *>(k + src + D / 2);
        const uint4 vx = *reinterpret_cast<const uint4 *>(v + src), vy = *reinterpret_cast<const uint4 *>(v + src + D / 2);
        if (!a.turned)
            rotate_halves<T>(x, y, cs, il);
        *reinterpret_cast<uint4 *>(pk + dst) = x;
        *reinterpret_cast<uint4 *>(pk + dst + D / 2) = y;
        *reinterpret_cast<uint4 *>(pv + dst) = vx;
        *reinterpret_cast<uint4 *>(pv + dst + D / 2) = vy;
    }
}

template <typename T, int D>
static cudaError_t append(PageArgs a, const PageTable &t, int n_sms, cudaStream_t s)
{
    constexpr int kTokens = kApThreads / (D / 2 / Vec<T>::N);
    const int units = a.n_layers * a.n_kv_heads;
    const int64_t tb = ((int64_t)a.total_q + kTokens - 1) / kTokens;
    a.per_cta = (int32_t)std::clamp<int64_t>(tb * units / (16 * (int64_t)n_sms), 1, std::min(units, 16));
    const int64_t grid = tb * ((units + a.per_cta - 1) / a.per_cta);
    return launch_pdl(k_page_append<T, D>, grid, kApThreads, 0, true, s, a, t);
}

cudaError_t launch_page_append(const PageArgs &a, const PageTable &t, int dtype, int head_dim, int n_sms, cudaStream_t s)
{
    if (dtype == KVR_DTYPE_BF16)
        return head_dim == 128 ? append<__nv_bfloat16, 128>(a, t, n_sms, s) : append<__nv_bfloat16, 64>(a, t, n_sms, s);
    return head_dim == 128 ? append<float, 128>(a, t, n_sms, s) : append<float, 64>(a, t, n_sms, s);
}

// ---------------------------------------------------------------------------
// packing
// ---------------------------------------------------------------------------
namespace {

constexpr int kPkWarps = 4;

// For scales near or below the smallest normal numbers, whose reciprocal may be no fp32 number.
__device__ __noinline__ uint32_t pack8_small(uint4 raw, float scale)
{
    float f[8];
    Vec<__nv_bfloat16>::get(raw, f);
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        w |= (uint32_t)((int)fminf(fmaxf(rintf(__fdiv_rn(f[e], scale)), -7.f), 7.f) + 8) << (4 * e);
    return w;
}

// Eight values (dims 8 c .. 8 c + 7 of a group) as nibbles code + 8, dims in order, and the
// scale of the group, whose other values are in the other three lanes of the quad.
//
// scale = bf16(max |x| / 7), code = x / scale rounded, halves to even.  x and scale have 8
// significant bits, so that a quotient is a half, or at least 2^-10 away from one: rounded
// to a multiple of 2^-11 first, x times the reciprocal (off by 2^-21 at most) is exactly
// the half or on the right side of it.  The codes are joined as fp32 integers (up to 2^16),
// which leaves the integer pipes to the rest.  (Divisions and conversions instead: 133 us
// for 2,592 rows, 112 units, packed and unpacked; 68 so.)
__device__ __forceinline__ uint32_t pack8(const uint4 &raw, uint16_t &scale_bits)
{
    const uint32_t x[4] = {raw.x, raw.y, raw.z, raw.w};
    // magnitudes as integers: a NaN or an infinity is above every number
    uint32_t top2 = __vmaxu2(__vmaxu2(x[0] & 0x7fff7fffu, x[1] & 0x7fff7fffu), __vmaxu2(x[2] & 0x7fff7fffu, x[3] & 0x7fff7fffu));
    top2 = __vmaxu2(top2, __shfl_xor_sync(0xffffffffu, top2, 1));
    top2 = __vmaxu2(top2, __shfl_xor_sync(0xffffffffu, top2, 2));
    const uint32_t top = max(top2 & 0xffffu, top2 >> 16);
    // (a seventh of an 8-bit number is nowhere near the middle of two: the product rounds as the quotient)
    const __nv_bfloat16 sb = __float2bfloat16_rn(__uint_as_float(top << 16) * (1.f / 7.f));
    const float scale = __bfloat162float(sb);
    const bool finite = top < 0x7f80u;
    scale_bits = finite ? __bfloat16_as_ushort(sb) : (uint16_t)0x7fff;   // NaN
    if (!finite || !(scale > 0.f))
        return 0x88888888u;
    if (scale < 1e-36f)
        return pack8_small(raw, scale);
    float f[8];
    Vec<__nv_bfloat16>::get(raw, f);
    const float inv = __frcp_rn(scale);
    constexpr float kGrid = 6144.f, kWhole = 12582912.f;   // 1.5 * 2^12, 2^23: a sum with them is rounded to 2^-11, to 1
#pragma unroll
    for (int e = 0; e < 8; ++e)
        f[e] = __fadd_rn(__fadd_rn(__fmaf_rn(f[e], inv, kGrid), kWhole - kGrid), -kWhole);
    // sum of 16^e (code + 8), four at a time
    const float a = fmaf(fmaf(f[3], 16.f, f[2]), 256.f, fmaf(f[1], 16.f, f[0])) + (34952.f + 8388608.f);
    const float b = fmaf(fmaf(f[7], 16.f, f[6]), 256.f, fmaf(f[5], 16.f, f[4])) + (34952.f + 8388608.f);
    return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x5410);
}

// nibbles 0..7 (dims in order) -> the keys' order: dim 2 m at m, dim 2 m + 1 at m + 4
__device__ __forceinline__ uint32_t spread_pairs(uint32_t w)
{
    // each step takes the middle two of four neighbours: halves of bytes, then bytes, ..
    uint32_t t = (w ^ (w >> 4)) & 0x00f000f0u;
    w ^= t ^ (t << 4);
    t = (w ^ (w >> 8)) & 0x0000ff00u;
    return w ^ t ^ (t << 8);
}

}  // namespace

// One warp: the keys or the values of one block of 32 rows, 8 at a time (a loop, which the
// instruction cache holds), the next 8 asked for ahead.  Lane 4 n + c holds, of row n of
// the 8, the dims 32 g + 8 c .. of every group g.  Packing 2,592 rows, 112 units, and
// restoring them: 381 MB in 68 us, 0.84 of the copy rate; packing alone issues an
// instruction in 0.8 of the cycles, restoring is bound by HBM.
template <bool kUnpack>
__global__ void __launch_bounds__(32 * kPkWarps)
    k_page_pack(const __grid_constant__ PageArgs a, const __grid_constant__ PageTable t, int64_t n_items)
{
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const DevPageReq *reqs = a.reqs ? a.reqs : t.reqs;
    const int32_t *ids = a.reqs ? a.ids : t.ids;
    const int lane = threadIdx.x & 31, n = lane >> 2, c = lane & 3;
    const int64_t item = (int64_t)blockIdx.x * kPkWarps + (threadIdx.x >> 5);
    if (item >= n_items)
        return;
    const int which = (int)(item & 1), units = a.n_layers * a.n_kv_heads;
    const int64_t blk = (item >> 1) / units;
    const int u = (int)((item >> 1) - blk * units), l = u / a.n_kv_heads, h = u - l * a.n_kv_heads;
    const DevPageReq &rq = reqs[request_of(reqs, a.n_reqs, (int)blk)];
    const int row = rq.pos0 + (int)(blk - rq.q_off) * kPackRows, pg = page_of(a, row), in = row - pg * a.g.rows;
    uint4 *x = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(which ? a.g.v : a.g.k) + (int64_t)page_id(rq, ids, pg) * a.g.s_page +
                                         l * a.g.s_layer + h * a.g.s_head + (int64_t)in * 128) + 16 * n + c;
    uint8_t *p = a.g.packed + packed_block(a, rq, ids, u, row);
    // a value word of octet c' is, transposed, that of lane 4 (lane & 7) + c'
    const int place = 16 * (which ? 4 * (lane & 7) + (lane >> 3) : lane);
    if constexpr (!kUnpack) {
        uint4 next[4];
#pragma unroll
        for (int g = 0; g < 4; ++g)
            next[g] = x[4 * g];
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
            uint4 raw[4];
#pragma unroll
            for (int g = 0; g < 4; ++g)
                raw[g] = next[g];
            if (i < 3)
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    next[g] = x[128 * (i + 1) + 4 * g];
            uint32_t w[4];
            uint16_t sc[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                w[g] = pack8(raw[g], sc[g]);
                w[g] = which ? transpose_nibbles(w[g], lane) : spread_pairs(w[g]);
            }
            *reinterpret_cast<uint4 *>(p + codes_at(i, which) + place) = make_uint4(w[0], w[1], w[2], w[3]);
            if (c == 0)
                *reinterpret_cast<uint2 *>(p + scales_at(8 * i + n, which)) =
                    make_uint2(sc[0] | (uint32_t)sc[1] << 16, sc[2] | (uint32_t)sc[3] << 16);
        }
    } else {
        uint4 codes[4];
        uint2 sc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            codes[i] = *reinterpret_cast<const uint4 *>(p + codes_at(i, which) + place);
            sc[i] = *reinterpret_cast<const uint2 *>(p + scales_at(8 * i + n, which));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w[4] = {codes[i].x, codes[i].y, codes[i].z, codes[i].w};
#pragma unroll
            for (int g = 0; g < 4; ++g)
                x[128 * i + 4 * g] = restore8(w[g], which, prmt(g < 2 ? sc[i].x : sc[i].y, 0u, (g & 1) ? 0x3232u : 0x1010u), lane);
        }
    }
}

cudaError_t launch_page_pack(const PageArgs &a, const PageTable &t, int64_t n_blocks, bool unpack, cudaStream_t s)
{
    const int64_t items = 2 * n_blocks * a.n_layers * a.n_kv_heads, grid = (items + kPkWarps - 1) / kPkWarps;
    if (grid == 0)
        return cudaSuccess;
    return launch_pdl(unpack ? k_page_pack<true> : k_page_pack<false>, grid, 32 * kPkWarps, 0, true, s, a, t, items);
}

// ---------------------------------------------------------------------------
// attention on the CUDA cores
// ---------------------------------------------------------------------------
namespace {
constexpr int kSmThreads = 256;
constexpr int kSmTeams = kSmThreads / 8;
}  // namespace

// One CTA: one token, up to kSmHeads (2 or 4) of the query heads of one kv head.  Teams of 8
// threads, D / 8 dims each, go through the visible keys by turns, every team with its own
// running maximum, sum and output; they are joined at the end.  Few CTAs are bound by a team's
// chain of loads, sums over its threads and exponentials, so a team takes four rows (of 128 fp32
// dims two) at once; many by instructions: without empty heads.  fp32, head_dim 64, 2 heads a kv
// head, 8 units: 4 x 1 token on 2,000 rows 22 us, 49 with a row at a time; 4 x 24 tokens 80 us,
// 150 with places for 4 heads, 171 with a row at a time too (bf16 81, 191 and 173): the reads alone
// are 5 us, but each token takes the whole cache again, and every product is an FMA (issue slots
// 57 % busy).  head_dim 128 32 and 172 us, its reads 10.  16 tokens on 193 rows, 2 units: 5.3 us in a
// replayed graph, the host's call 8 to 10.
template <typename T, int D, int kSmHeads>
__global__ void __launch_bounds__(kSmThreads)
    k_page_simt(const __grid_constant__ PageArgs a, const __grid_constant__ PageTable t)
{
    constexpr int N = D / 8, V = Vec<T>::N;   // dims of a thread: vectors 8 i + j of a row, i < N / V
    constexpr int kKeys = N / V > 2 ? 2 : 4;
    __shared__ float qs[kSmHeads][D];
    __shared__ float st_m[kSmTeams][kSmHeads], st_l[kSmTeams][kSmHeads];
    __shared__ float st_o[kSmTeams][D];
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const DevPageReq *reqs = a.reqs ? a.reqs : t.reqs;
    const int32_t *ids = a.reqs ? a.ids : t.ids;
    const int G = a.n_q_heads / a.n_kv_heads, hc = (G + kSmHeads - 1) / kSmHeads;
    int64_t b = blockIdx.x;
    const int g0 = (int)(b % hc) * kSmHeads, nh = min(kSmHeads, G - g0);
    b /= hc;
    const int h = (int)(b % a.n_kv_heads);
    b /= a.n_kv_heads;
    const int tok = (int)(b % a.total_q), l = (int)(b / a.total_q);
    const DevPageReq &rq = reqs[request_of(reqs, a.n_reqs, tok)];
    const int pos = rq.pos0 + tok - rq.q_off;
    const int64_t q0 = (((int64_t)l * a.total_q + tok) * a.n_q_heads + h * G + g0) * D;
    const T *q = static_cast<const T *>(a.q) + q0;
    const bool il = a.interleaved != 0;
    for (int i = threadIdx.x; i < nh * (D / 2); i += kSmThreads) {
        const int g = i / (D / 2), pr = i % (D / 2), d0 = il ? 2 * pr : pr, d1 = il ? 2 * pr + 1 : pr + D / 2;
        const float2 cs = rope_cs(a.rope, D / 2, pos, pr);
        const float x = (float)q[g * D + d0], y = (float)q[g * D + d1];
        qs[g][d0] = fmaf(x, cs.x, -(y * cs.y)) * a.scale_log2;
        qs[g][d1] = fmaf(x, cs.y, y * cs.x) * a.scale_log2;
    }
    __syncthreads();
    const int team = threadIdx.x >> 3, j = threadIdx.x & 7;
    const Sees see = sees(a, rq, pos);
    const int lo = min(see.lo, see.hi), few = min(see.few, see.hi), n_keys = few + see.hi - lo;
    float qr[kSmHeads][N], o[kSmHeads][N], m[kSmHeads], ls[kSmHeads];
#pragma unroll
    for (int g = 0; g < kSmHeads; ++g) {
        m[g] = -INFINITY;
        ls[g] = 0.f;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            o[g][e] = 0.f;
            qr[g][e] = g < nh ? qs[g][(8 * (e / V) + j) * V + e % V] : 0.f;
        }
    }
    const uint32_t team_mask = 0xffu << (8 * ((threadIdx.x >> 3) & 3));
    // kKeys rows at a time: their loads and their scores' sums do not wait for each other
    for (int i = team; i < n_keys; i += kKeys * kSmTeams) {
        uint4 kv[kKeys][N / V], vv[kKeys][N / V];
#pragma unroll
        for (int u = 0; u < kKeys; ++u) {
            const int r = min(i + u * kSmTeams, n_keys - 1), row = r < few ? r : lo + r - few, pg = page_of(a, row);
            const int64_t at = (int64_t)page_id(rq, ids, pg) * a.g.s_page + l * a.g.s_layer + h * a.g.s_head +
                               (int64_t)(row - pg * a.g.rows) * D;
            const uint4 *kp = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.g.k) + at);
            const uint4 *vp = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.g.v) + at);
#pragma unroll
            for (int e = 0; e < N / V; ++e) {
                kv[u][e] = __ldg(kp + 8 * e + j);
                vv[u][e] = __ldg(vp + 8 * e + j);
            }
        }
        float s[kSmHeads][kKeys];
#pragma unroll
        for (int u = 0; u < kKeys; ++u) {
            float f[N];
#pragma unroll
            for (int e = 0; e < N / V; ++e)
                Vec<T>::get(kv[u][e], f + V * e);
#pragma unroll
            for (int g = 0; g < kSmHeads; ++g) {
                float x = 0.f;
#pragma unroll
                for (int e = 0; e < N; ++e)
                    x = fmaf(qr[g][e], f[e], x);
                s[g][u] = x;
            }
        }
#pragma unroll
        for (int d = 1; d <= 4; d <<= 1)
#pragma unroll
            for (int u = 0; u < kKeys; ++u)
#pragma unroll
                for (int g = 0; g < kSmHeads; ++g)
                    s[g][u] += __shfl_xor_sync(team_mask, s[g][u], d);
#pragma unroll
        for (int g = 0; g < kSmHeads; ++g) {
            float mn = m[g];
#pragma unroll
            for (int u = 0; u < kKeys; ++u) {
                if (i + u * kSmTeams >= n_keys)   // (the last row again)
                    s[g][u] = -INFINITY;
                mn = fmaxf(mn, s[g][u]);
            }
            const float corr = mn == -INFINITY ? 1.f : exp2f(m[g] - mn);
            m[g] = mn;
            ls[g] *= corr;
#pragma unroll
            for (int e = 0; e < N; ++e)
                o[g][e] *= corr;
#pragma unroll
            for (int u = 0; u < kKeys; ++u) {
                s[g][u] = mn == -INFINITY ? 0.f : exp2f(s[g][u] - mn);
                ls[g] += s[g][u];
            }
        }
#pragma unroll
        for (int u = 0; u < kKeys; ++u) {
            float f[N];
#pragma unroll
            for (int e = 0; e < N / V; ++e)
                Vec<T>::get(vv[u][e], f + V * e);
#pragma unroll
            for (int g = 0; g < kSmHeads; ++g)
#pragma unroll
                for (int e = 0; e < N; ++e)
                    o[g][e] = fmaf(s[g][u], f[e], o[g][e]);
        }
    }
    if (j == 0) {
#pragma unroll
        for (int g = 0; g < kSmHeads; ++g) {
            st_m[team][g] = m[g];
            st_l[team][g] = ls[g];
        }
    }
#pragma unroll
    for (int g = 0; g < kSmHeads; ++g) {
        if (g >= nh)
            break;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < N; ++e)
            st_o[team][(8 * (e / V) + j) * V + e % V] = o[g][e];
        __syncthreads();
        float M = -INFINITY, L = 0.f;
        for (int w = 0; w < kSmTeams; ++w)
            M = fmaxf(M, st_m[w][g]);
        for (int d = threadIdx.x; d < D; d += kSmThreads) {
            float x = 0.f;
            L = 0.f;
            for (int w = 0; w < kSmTeams; ++w) {
                const float f = st_m[w][g] == -INFINITY ? 0.f : exp2f(st_m[w][g] - M);
                L = fmaf(st_l[w][g], f, L);
                x = fmaf(st_o[w][d], f, x);
            }
            // a row that sees no key is zero; one that does has a denominator of at least 1,
            // or a NaN or an infinity in its query or a key
            if (n_keys > 0 && !(L > 0.f && L < INFINITY) && d == 0)
                atomicCAS(a.err, kDevOk, kDevBadInput);
            T *out = static_cast<T *>(a.out) + q0 + g * D;
            out[d] = (T)(n_keys > 0 ? x / L : 0.f);
        }
    }
}

template <typename T, int D>
static cudaError_t simt(const PageArgs &a, const PageTable &t, cudaStream_t s)
{
    const int G = a.n_q_heads / a.n_kv_heads, heads = G <= 2 ? 2 : 4;
    const int64_t grid = (int64_t)a.n_layers * a.total_q * a.n_kv_heads * ((G + heads - 1) / heads);
    return launch_pdl(heads == 2 ? k_page_simt<T, D, 2> : k_page_simt<T, D, 4>, grid, kSmThreads, 0, true, s, a, t);
}

cudaError_t launch_page_simt(const PageArgs &a, const PageTable &t, int dtype, int head_dim, cudaStream_t s)
{
    if (dtype == KVR_DTYPE_BF16)   // (head_dim 128: the tensor-core kernels)
        return head_dim == 64 ? simt<__nv_bfloat16, 64>(a, t, s) : cudaErrorInvalidValue;
    return head_dim == 128 ? simt<float, 128>(a, t, s) : simt<float, 64>(a, t, s);
}

}  // namespace kvr
