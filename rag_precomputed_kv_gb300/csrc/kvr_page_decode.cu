// kvr_page_decode.cu -- attention of a few query rows over a paged cache, whose
// older rows may be packed to 4 bits (bf16, head_dim 128).
//
//     o_r = sum_j e^{s_rj} v_j / sum_j e^{s_rj},   s_rj = scale <q_r, k_j>,
// over the rows j that query row r sees, r = (token, query head of the kv head),
// up to 16 rows a request.  Every key and value is read once; the kernel is
// bound by these reads, 512 bytes a row and (layer, kv-head), 144 where packed.
//
// One CTA, or a cluster of 2 to 8 where (request, unit) pairs are few, takes one
// request's (layer, kv-head).  Its warps go through the visible key tiles by
// turns, each with its own two-stage ring filled by cp.async (16 bf16 rows, or 64
// packed ones, a stage: any page size and stride, rows that are not there are
// zeros) and its own running maximum, sum and output in registers; no warp waits
// for another before the states are joined, in a fixed order, through shared
// memory and the cluster's.  Three CTAs of four warps are resident on an SM.
//
// Both products are warp MMAs (mma.sync m16n8k16; at 16 rows a tcgen05 MMA would
// pass every tile through TMEM).  Packed rows are not restored to bf16 rows: a
// nibble n under the exponent bits of 128 is the bf16 number 128 + n, and
//   keys    sum_d q_d (n_d + 128) - 136 sum_d q_d = sum_d q_d code_d: the second
//           term is where the accumulator starts; the group's fp32 result is then
//           scaled and added, so that a score has the codes' and scales' exact
//           values in it;
//   values  the (row, group) scale goes to the probability, rounded to bf16 once
//           with it, and 136 is subtracted from the operand, which is exact.
// Rounded to bf16: the turned queries and the (scaled) probabilities, because
// they are operands of products with bf16 numbers.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "kvr_decode_common.cuh"
#include "kvr_page_common.cuh"

namespace kvr {

namespace {

using namespace page;
using dec::dec_ex2;
using dec::dec_smem_u32;
using dec::ldsm_x4_t;
using dec::mma_bf16;
using dec::pack2;

constexpr int kPdWarps = 4;
constexpr int kPdThreads = 32 * kPdWarps;
constexpr int kPdKeys = 16, kPdPacked = 64;          // rows of a tile
constexpr int kPdStage = 2 * kPackBytes;             // 64 packed rows, or 16 bf16 keys and values (8,192)
constexpr int kPdRing = 2 * kPdStage;
constexpr int kPdSmem = kPdWarps * kPdRing;
constexpr int kPdCtas = 3;                           // resident on an SM
constexpr int kPdPitch = 136;                        // floats of a row of a warp's output (no bank conflicts)
static_assert(16 * kPdPitch * 4 + 128 <= kPdStage && 16 * 128 * 4 + 128 <= kPdStage, "states over the ring");

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ float4 ld_cluster(uint32_t a)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ float ld_cluster1(uint32_t a)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t at_rank(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_meet()
{
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Nibbles 0 and 4 of w as the bf16 pair (128 + nibble).
__device__ __forceinline__ uint32_t pair128(uint32_t w) { return (w & 0x000f000fu) | 0x43004300u; }
// 136 less, exactly.
__device__ __forceinline__ uint32_t less136(uint32_t w)
{
    const uint32_t c = 0x43084308u;
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&w), *reinterpret_cast<const __nv_bfloat162 *>(&c));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// d = a b + c
__device__ __forceinline__ void mma_from(float *d, const uint32_t *a, uint32_t b0, uint32_t b1, float c0, float c2)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %11, %11};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c2));
}

// The tiles that some query of a request meets: packed ones of 64 rows, then bf16
// ones of 16; of each the first rows', then the window's.
struct TileList {
    int t0[4], n[4];
    int lo, hi, few, body;

    __host__ __device__ __forceinline__ void set(const DevPageReq &r, int window, int n_first)
    {
        hi = r.kv_len < r.pos0 + r.q_len ? r.kv_len : r.pos0 + r.q_len;
        lo = window > 0 && r.pos0 - window + 1 > 0 ? r.pos0 - window + 1 : 0;
        lo = lo < hi ? lo : hi;
        few = n_first < lo ? n_first : lo;
        body = r.packed_len;
        auto part = [](int a, int b, int size, int from, int &first, int &count) {   // tiles of rows [a, b), from `from` on
            first = a / size > from ? a / size : from;
            const int end = a < b ? (b + size - 1) / size : 0;
            count = end > first ? end - first : 0;
        };
        const int hp = hi < body ? hi : body, fp = few < body ? few : body, lb = lo > body ? lo : body;
        part(0, fp, kPdPacked, 0, t0[0], n[0]);
        part(lo, hp, kPdPacked, n[0], t0[1], n[1]);
        part(body, few, kPdKeys, 0, t0[2], n[2]);
        part(lb, hi, kPdKeys, t0[2] + n[2], t0[3], n[3]);
    }
    __host__ __device__ __forceinline__ int total() const { return n[0] + n[1] + n[2] + n[3]; }
    __device__ __forceinline__ bool seen(int j) const { return j < hi && (j >= lo || j < few); }
    __device__ __forceinline__ bool block_seen(int j) const { return j < body && (j < few || (j < hi && j + kPackRows > lo)); }
    // tile i: its first row, and whether it is packed
    __device__ __forceinline__ int row(int i, bool &packed) const
    {
        const int p = n[0] + n[1];
        packed = i < p;
        if (packed)
            return (i < n[0] ? t0[0] + i : t0[1] + i - n[0]) * kPdPacked;
        return (i < p + n[2] ? t0[2] + i - p : t0[3] + i - p - n[2]) * kPdKeys;
    }
};

}  // namespace

__global__ void __launch_bounds__(kPdThreads, kPdCtas)
    k_page_decode(const __grid_constant__ PageArgs a, const __grid_constant__ PageTable t, int n_ctas)
{
    extern __shared__ __align__(128) uint8_t pd_smem[];
    pdl_wait_prerequisites();   // (also before leaving: the next kernel's wait stands for those before this one)
    pdl_launch_dependents();
    const DevPageReq *reqs = a.reqs ? a.reqs : t.reqs;
    const int32_t *ids = a.reqs ? a.ids : t.ids;
    const int G = a.n_q_heads / a.n_kv_heads;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = lane >> 2, c = lane & 3;
    const uint32_t rank = blockIdx.x % (unsigned)n_ctas;
    const int item = (int)(blockIdx.x / (unsigned)n_ctas), u = item / a.n_reqs, l = u / a.n_kv_heads, h = u - l * a.n_kv_heads;
    const DevPageReq rq = reqs[item - u * a.n_reqs];
    const int rows = rq.q_len * G;
    if (rows == 0 || rows > kPageFewRows)
        return;   // (all CTAs of the cluster)
    TileList tl;
    tl.set(rq, a.window, a.n_first);
    const int n_t = tl.total(), step = kPdWarps * n_ctas;
    const int64_t unit = l * a.g.s_layer + h * a.g.s_head;
    const __nv_bfloat16 *gk = static_cast<const __nv_bfloat16 *>(a.g.k), *gv = static_cast<const __nv_bfloat16 *>(a.g.v);
    const uint32_t ring = dec_smem_u32(pd_smem) + (uint32_t)(warp * kPdRing);
    const bool one_page = a.g.rows % kPdKeys == 0;   // a tile's rows are in one page

    auto issue = [&](int i, int stage) {
        if (i < n_t) {
            bool packed;
            const int r0 = tl.row(i, packed);
            const uint32_t dst = ring + (uint32_t)(stage * kPdStage);
            if (packed) {
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (tl.block_seen(r0 + k * kPackRows)) {
                        const uint8_t *src = a.g.packed + packed_block(a, rq, ids, u, r0 + k * kPackRows) + 16 * lane;
#pragma unroll
                        for (int x = 0; x < kPackBytes / 512; ++x)
                            copy16(dst + (uint32_t)(k * kPackBytes + 16 * lane + 512 * x), src + 512 * x, true);
                    }
            } else {
                const int ch = lane & 15;
                int64_t base = 0;
                if (one_page) {
                    const int pg = r0 / a.g.rows;
                    base = (int64_t)page_id(rq, ids, pg) * a.g.s_page + unit + (int64_t)(r0 - pg * a.g.rows) * 128;
                }
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const int r = (lane >> 4) + 2 * x, j = r0 + r;
                    const bool there = tl.seen(j);
                    int64_t at = base + r * 128;
                    if (!one_page && there) {
                        const int pg = j / a.g.rows;
                        at = (int64_t)page_id(rq, ids, pg) * a.g.s_page + unit + (int64_t)(j - pg * a.g.rows) * 128;
                    }
                    at = there ? at + 8 * ch : 0;
                    copy16(dst + (uint32_t)(r * 256 + ((ch ^ ((r & 1) << 2)) << 4)), gk + at, there);
                    copy16(dst + (uint32_t)(4096 + r * 256 + ((ch ^ (r & 7)) << 4)), gv + at, there);
                }
            }
        }
        copies_end();
    };
    int it = (int)rank * kPdWarps + warp;
    issue(it, 0);
    issue(it + step, 1);

    // Q as the A operand: rows n and n + 8, of group g the dims 32 g + 8 c + 0..7, pair
    // m at step m / 2; turned by the rows' positions
    uint32_t qa[4][2][4];
    float start[4][2];   // -136 times a group's sum
    {
        const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) +
                                 (((int64_t)l * a.total_q + rq.q_off) * a.n_q_heads + h * G) * 128 + 8 * c;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int r = n + 8 * x, tok = r / G;
            const bool some = r < rows;
            uint4 v[4];
#pragma unroll
            for (int g = 0; g < 4; ++g)
                v[g] = some ? *reinterpret_cast<const uint4 *>(q + ((int64_t)tok * a.n_q_heads + (r - tok * G)) * 128 + 32 * g)
                            : make_uint4(0, 0, 0, 0);
            if (some) {
                const int pos = rq.pos0 + tok;
                float cs[8], sn[8];
                if (a.interleaved) {
#pragma unroll
                    for (int g = 0; g < 4; g += 2) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float2 w = rope_cs(a.rope, 64, pos, 16 * (g + (e >> 2)) + 4 * c + (e & 3));
                            cs[e] = w.x;
                            sn[e] = w.y;
                        }
                        rotate_bf16x8_il(v[g], v[g + 1], cs, sn);
                    }
                } else {
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float2 w = rope_cs(a.rope, 64, pos, 32 * g + 8 * c + e);
                            cs[e] = w.x;
                            sn[e] = w.y;
                        }
                        rotate_bf16x8(v[g], v[g + 2], cs, sn);
                    }
                }
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const uint32_t w[4] = {v[g].x, v[g].y, v[g].z, v[g].w};
                float s = 0.f;
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    qa[g][m >> 1][2 * (m & 1) + x] = w[m];
                    s += bf_lo(w[m]) + bf_hi(w[m]);
                }
                s += __shfl_xor_sync(0xffffffffu, s, 1);
                s += __shfl_xor_sync(0xffffffffu, s, 2);
                start[g][x] = -136.f * s;
            }
        }
    }
    Sees see[2];
    int p_last = rq.pos0 + rq.q_len - 1;
#pragma unroll
    for (int x = 0; x < 2; ++x)
        see[x] = sees(a, rq, min(p_last, rq.pos0 + (n + 8 * x) / G));
    // rows that every query sees: below, and from (or among the first) on
    const int all_hi = min(rq.kv_len, rq.pos0 + 1), all_lo = a.window > 0 ? p_last - a.window + 1 : 0;

    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
    float o[16][4];
#pragma unroll
    for (int j = 0; j < 16; ++j)
        o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;

    // scores of 8 NT rows from row0 on become probabilities, O and l are brought to the
    // maximum they are relative to.  It moves only when it grows by more than 8 (log2),
    // which bf16 and fp32 hold, and a row's quad agrees on it.
    auto softmax = [&](float (*s)[4], auto nt, int row0) {
        constexpr int NT = decltype(nt)::value;
        const float sc = a.scale_log2;
        if (row0 + 8 * NT <= all_hi && (row0 >= all_lo || row0 + 8 * NT <= a.n_first)) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[i][e] *= sc;
        } else {
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[i][e] = see[e >> 1](row0 + 8 * i + 2 * c + (e & 1)) ? s[i][e] * sc : -INFINITY;
        }
        float corr[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            float mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < NT; ++i)
                mx = fmaxf(mx, fmaxf(s[i][2 * x], s[i][2 * x + 1]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            corr[x] = 1.f;
            if (mx > m_run[x] + 8.f) {
                corr[x] = dec_ex2(m_run[x] - mx);
                m_run[x] = mx;
            }
        }
        if (__any_sync(0xffffffffu, corr[0] != 1.f || corr[1] != 1.f)) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                o[j][0] *= corr[0];
                o[j][1] *= corr[0];
                o[j][2] *= corr[1];
                o[j][3] *= corr[1];
            }
            l_run[0] *= corr[0];
            l_run[1] *= corr[1];
        }
        const float nm[2] = {m_run[0] == -INFINITY ? 0.f : -m_run[0], m_run[1] == -INFINITY ? 0.f : -m_run[1]};
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[i][e] = dec_ex2(s[i][e] + nm[e >> 1]);
                l_run[e >> 1] += s[i][e];
            }
    };

    for (int stage = 0; it < n_t; it += step, stage ^= 1) {
        copies_wait<1>();
        __syncwarp();
        bool packed;
        const int row0 = tl.row(it, packed);
        const uint32_t st = ring + (uint32_t)(stage * kPdStage);
        if (packed) {
#pragma unroll 1
            for (int k = 0; k < 2; ++k) {
                const int r = row0 + k * kPackRows;
                if (!tl.block_seen(r))
                    continue;
                const uint32_t kb = st + (uint32_t)(k * kPackBytes), vb = kb + kPackHalf;
                float s[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 code = lds128(kb + 512 * i + 16 * lane), sc = lds128(kb + 2048 + 64 * i + 16 * c);
                    const uint32_t w[4] = {code.x, code.y, code.z, code.w}, s0[2] = {sc.x, sc.y}, s1[2] = {sc.z, sc.w};
                    s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        float d[4];
                        mma_from(d, qa[g][0], pair128(w[g]), pair128(w[g] >> 4), start[g][0], start[g][1]);
                        mma_bf16(d, qa[g][1], pair128(w[g] >> 8), pair128(w[g] >> 12));
                        const float x0 = (g & 1) ? bf_hi(s0[g >> 1]) : bf_lo(s0[g >> 1]);
                        const float x1 = (g & 1) ? bf_hi(s1[g >> 1]) : bf_lo(s1[g >> 1]);
                        s[i][0] = fmaf(x0, d[0], s[i][0]);
                        s[i][1] = fmaf(x1, d[1], s[i][1]);
                        s[i][2] = fmaf(x0, d[2], s[i][2]);
                        s[i][3] = fmaf(x1, d[3], s[i][3]);
                    }
                }
                softmax(s, std::integral_constant<int, 4>(), r);
                // rows that no query sees may have scales of NaN
                const bool whole = r + kPackRows <= tl.hi && (r >= tl.lo || r + kPackRows <= tl.few);
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    const uint4 c0 = lds128(vb + 512 * i + 16 * lane), c1 = lds128(vb + 512 * i + 512 + 16 * lane);
                    uint4 z0 = lds128(vb + 2048 + 64 * i + 16 * c), z1 = lds128(vb + 2048 + 64 * i + 64 + 16 * c);
                    if (!whole) {
                        const int j = r + 8 * i + 2 * c;
                        if (!tl.seen(j))
                            z0.x = z0.y = 0u;
                        if (!tl.seen(j + 1))
                            z0.z = z0.w = 0u;
                        if (!tl.seen(j + 8))
                            z1.x = z1.y = 0u;
                        if (!tl.seen(j + 9))
                            z1.z = z1.w = 0u;
                    }
                    const uint32_t w0[4] = {c0.x, c0.y, c0.z, c0.w}, w1[4] = {c1.x, c1.y, c1.z, c1.w};
                    const uint32_t s00[2] = {z0.x, z0.y}, s01[2] = {z0.z, z0.w}, s10[2] = {z1.x, z1.y}, s11[2] = {z1.z, z1.w};
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const float x00 = (g & 1) ? bf_hi(s00[g >> 1]) : bf_lo(s00[g >> 1]);
                        const float x01 = (g & 1) ? bf_hi(s01[g >> 1]) : bf_lo(s01[g >> 1]);
                        const float x10 = (g & 1) ? bf_hi(s10[g >> 1]) : bf_lo(s10[g >> 1]);
                        const float x11 = (g & 1) ? bf_hi(s11[g >> 1]) : bf_lo(s11[g >> 1]);
                        const uint32_t pa[4] = {pack2(s[i][0] * x00, s[i][1] * x01), pack2(s[i][2] * x00, s[i][3] * x01),
                                                pack2(s[i + 1][0] * x10, s[i + 1][1] * x11),
                                                pack2(s[i + 1][2] * x10, s[i + 1][3] * x11)};
#pragma unroll
                        for (int m = 0; m < 4; ++m)
                            mma_bf16(o[4 * g + m], pa, less136(pair128(w0[g] >> (4 * m))), less136(pair128(w1[g] >> (4 * m))));
                    }
                }
            }
        } else {
            float s[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const uint4 w = lds128(st + (uint32_t)((8 * i + n) * 256 + (((4 * g + c) ^ ((n & 1) << 2)) << 4)));
                    mma_bf16(s[i], qa[g][0], w.x, w.y);
                    mma_bf16(s[i], qa[g][1], w.z, w.w);
                }
            }
            softmax(s, std::integral_constant<int, 2>(), row0);
            const uint32_t pa[4] = {pack2(s[0][0], s[0][1]), pack2(s[0][2], s[0][3]), pack2(s[1][0], s[1][1]), pack2(s[1][2], s[1][3])};
            const int key = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
                uint32_t b0, b1, b2, b3;
                ldsm_x4_t(st + (uint32_t)(4096 + key * 256 + (((j + (lane >> 4)) ^ (key & 7)) << 4)), b0, b1, b2, b3);
                mma_bf16(o[j], pa, b0, b1);
                mma_bf16(o[j + 1], pa, b2, b3);
            }
        }
        __syncwarp();
        issue(it + 2 * step, stage);
    }
    copies_wait<0>();
    __syncwarp();

    // the warp's state over its ring
    auto area = [&](int w) { return reinterpret_cast<float *>(pd_smem + w * kPdRing); };
    {
        float *f = area(warp);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            l_run[x] += __shfl_xor_sync(0xffffffffu, l_run[x], 1);
            l_run[x] += __shfl_xor_sync(0xffffffffu, l_run[x], 2);
            if (c == 0) {
                f[16 * kPdPitch + n + 8 * x] = m_run[x];
                f[16 * kPdPitch + 16 + n + 8 * x] = l_run[x];
            }
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            *reinterpret_cast<float2 *>(f + n * kPdPitch + 8 * j + 2 * c) = make_float2(o[j][0], o[j][1]);
            *reinterpret_cast<float2 *>(f + (n + 8) * kPdPitch + 8 * j + 2 * c) = make_float2(o[j][2], o[j][3]);
        }
    }
    __syncthreads();
    // thread 32 k + i: rows k, k + 4, .., columns 4 i .. 4 i + 3
    auto write = [&](int r, int col, float M, float L, float4 v) {
        const int tok = r / G, pos = rq.pos0 + tok;
        const Sees s = sees(a, rq, pos);
        const bool some = s.hi > 0 && (s.few > 0 || s.lo < s.hi);
        // a NaN or an infinity in the query or a key leaves no finite positive denominator
        if (some && col == 0 && !(L > 0.f && L < INFINITY))
            atomicCAS(a.err, kDevOk, kDevBadInput);
        const float inv = some ? 1.f / L : 0.f;
        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.out) +
                             (((int64_t)l * a.total_q + rq.q_off + tok) * a.n_q_heads + h * G + (r - tok * G)) * 128 + col;
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack2(v.x * inv, v.y * inv), pack2(v.z * inv, v.w * inv));
    };
    const int col = 4 * lane;
    float *joined = reinterpret_cast<float *>(pd_smem + kPdStage);   // behind warp 0's state: [16][128], 16 maxima, 16 sums
    for (int r = warp; r < rows; r += kPdWarps) {
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < kPdWarps; ++w)
            M = fmaxf(M, area(w)[16 * kPdPitch + r]);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kPdWarps; ++w) {
            const float mw = area(w)[16 * kPdPitch + r], f = mw == -INFINITY ? 0.f : dec_ex2(mw - M);
            const float4 x = *reinterpret_cast<const float4 *>(area(w) + r * kPdPitch + col);
            // (a warp whose scores were NaN has a NaN sum under a maximum of -inf)
            L += mw == -INFINITY ? area(w)[16 * kPdPitch + 16 + r] : area(w)[16 * kPdPitch + 16 + r] * f;
            v.x = fmaf(x.x, f, v.x);
            v.y = fmaf(x.y, f, v.y);
            v.z = fmaf(x.z, f, v.z);
            v.w = fmaf(x.w, f, v.w);
        }
        if (n_ctas == 1) {
            write(r, col, M, L, v);
        } else {
            *reinterpret_cast<float4 *>(joined + r * 128 + col) = v;
            if (lane == 0) {
                joined[16 * 128 + r] = M;
                joined[16 * 128 + 16 + r] = L;
            }
        }
    }
    if (n_ctas == 1)
        return;
    cluster_meet();
    const uint32_t mine = dec_smem_u32(joined);
    for (int r = (int)rank + n_ctas * warp; r < rows; r += n_ctas * kPdWarps) {
        float M = -INFINITY, L = 0.f;
        for (int k = 0; k < n_ctas; ++k)
            M = fmaxf(M, ld_cluster1(at_rank(mine + 4u * (uint32_t)(16 * 128 + r), (uint32_t)k)));
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < n_ctas; ++k) {
            const float mk = ld_cluster1(at_rank(mine + 4u * (uint32_t)(16 * 128 + r), (uint32_t)k));
            const float lk = ld_cluster1(at_rank(mine + 4u * (uint32_t)(16 * 128 + 16 + r), (uint32_t)k));
            const float4 x = ld_cluster(at_rank(mine + 4u * (uint32_t)(r * 128 + col), (uint32_t)k));
            const float f = mk == -INFINITY ? 0.f : dec_ex2(mk - M);
            L += mk == -INFINITY ? lk : lk * f;
            v.x = fmaf(x.x, f, v.x);
            v.y = fmaf(x.y, f, v.y);
            v.z = fmaf(x.z, f, v.z);
            v.w = fmaf(x.w, f, v.w);
        }
        write(r, col, M, L, v);
    }
    cluster_meet();   // a CTA's state is read by the others until here
}

cudaError_t launch_page_decode(const PageArgs &a, const PageTable &t, const DevPageReq *host_reqs, int n_sms, cudaStream_t s)
{
    static std::atomic<bool> attr_set[64] = {};   // per device (host threads may race: same value)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev >= 64 || !attr_set[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(k_page_decode, cudaFuncAttributeMaxDynamicSharedMemorySize, kPdSmem);
        if (e != cudaSuccess)
            return e;
        if (dev < 64)
            attr_set[dev].store(true, std::memory_order_release);
    }
    const int units = a.n_layers * a.n_kv_heads, G = a.n_q_heads / a.n_kv_heads;
    int64_t few = 0;
    int most = 0;
    for (int b = 0; b < a.n_reqs; ++b) {
        if (host_reqs[b].q_len == 0 || host_reqs[b].q_len * (int64_t)G > kPageFewRows)
            continue;
        TileList tl;
        tl.set(host_reqs[b], a.window, a.n_first);
        most = std::max(most, tl.total());
        ++few;
    }
    if (few == 0)
        return cudaSuccess;
    // as many CTAs of a (request, unit) as are resident at once, each warp with two tiles at least
    int c = 1;
    while (c < 8 && few * units * c * 2 <= (int64_t)kPdCtas * n_sms && most >= 2 * kPdWarps * 2 * c)
        c *= 2;
    return launch_cluster(k_page_decode, (int64_t)a.n_reqs * units * c, kPdThreads, kPdSmem, c, s, a, t, c);
}

}  // namespace kvr
