// kvr_page_decode.cu -- attention of a few query rows over a paged cache, whose
// older rows may be packed to 4 bits (bf16, head_dim 128).
//
//     o_r = sum_j e^{s_rj} v_j / sum_j e^{s_rj},   s_rj = scale <q_r, k_j>,
// over the rows j that query row r sees, r = (token, query head of the kv head),
// up to 16 rows a request.  Every key and value is read once; the kernel is
// bound by these reads, 512 bytes a row and (layer, kv-head), 144 where packed.
//
// One CTA, or a cluster of 2 to 8 where (request, unit) pairs are few, takes one
// request's (layer, kv-head).  Its warps go through the visible key tiles by turns, each
// with its own ring filled by cp.async (tiles of 16 bf16 or 32 packed rows: any page size
// and stride, rows that are not there are zeros) and its own running maximum, sum and
// output in registers; no warp waits for another before the states are joined, in a
// fixed order, through shared memory and the cluster's.  Three CTAs of four warps are
// resident on an SM, four in calls with packed rows.
//
// Both products are warp MMAs (mma.sync m16n8k16; at 16 rows a tcgen05 MMA would
// pass every tile through TMEM), with keys and values as the 16-row operand and the
// query rows, eight at a time, as the columns: S^T = K Q^T and O^T = V^T P^T, so that
// a step of up to 8 query heads a kv head does half of what 16 rows would take.
// The probabilities change from the one's layout to the other's by movmatrix.
// Packed rows are not restored to bf16 rows:
//   keys    as fp16 bits a nibble n is the number n 2^-24, and 16 n 2^-24 four bits
//           higher (fp16 numbers are their bits' multiples of 2^-24 up to 2,047), which
//           the MMA takes exactly.  sum_d q_d n_d - 8 sum_d q_d = sum_d q_d code_d: the
//           second term is where the accumulator starts.  The group's fp32 result is then
//           scaled and added, so that a score has the codes' and scales' exact values;
//   values  a nibble n under the exponent bits of 128 is 128 + n in bf16, and 136 is
//           subtracted, which is exact; the (row, group) scale goes to the probability,
//           rounded to bf16 once with it.
// Queries and probabilities that meet bf16 rows are two bf16 terms each (16 bits): the
// memory's pace leaves room for that, and the output is off by its own rounding alone
// (0.0017 of its norm; 0.0029 with one term each).  Queries that meet packed rows are fp16
// times a power of two of their row, the largest element between 2^12 and 2^13 (11 bits of
// an element, fewer below 2^-22 of the largest or 2^-114); probabilities there are rounded to
// bf16 (0.0024), as a second term would be half as many products again in the step's chain.
//
// Measured: 4 x 2,656 bf16 rows, 112 units 93 us (6.5 TB/s); 8 windows of 4,100 rows, 256
// units 600 us (7.1 TB/s; reads alone run above the copy rate).  33,280 packed rows, 256
// units 271 to 293 us, 4.2 to 4.6 TB/s: no pipe is full (issue slots and ALU 0.58 of the time, half
// of it with extracting codes, DRAM 0.49); what bounds it is the length of a step's chain, codes,
// products, exponentials, products, at a fifth of the warps that an SM can hold.  On the way there (33,280 packed rows): the 16 query rows as the MMA's
// rows 699 us; as columns, eight at a time 374; steps of 16 rows in a loop that the
// instruction cache holds, scales of a step together 348 (not a loop, 16 x 1,216 rows take
// 240 us, 197 as one); four CTAs an SM 317; keys as subnormal numbers (one shift a word
// instead of three) 286; both products of a group in one accumulator, the upper nibbles'
// queries a sixteenth 269.  Shifts as high products of the multiplier, which is idle: 299
// against 286.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

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
constexpr int kPdKeys = 16, kPdPacked = kPackRows;   // rows of a tile
constexpr int kPdKeyBytes = kPdKeys * 2 * 256;
constexpr int kPdPitch = 132;                        // floats of a row of a warp's output (two rows 8 banks apart)

// A warp's ring.  Calls without packed rows: two tiles of 16 rows, three CTAs on an
// SM.  Calls with them: three packed tiles, in whose place the bf16 ones behind them come one
// at a time; up to 8 query rows leave registers for four CTAs on an SM.
template <int NR, bool kPack>
struct Ring {
    static constexpr int kCtas = kPack && NR == 1 ? 4 : 3;
    static constexpr int kPackStages = 3, kKeyStages = kPack ? 1 : 2;
    static constexpr int kBytes = kPack ? kPackStages * kPackBytes : kKeyStages * kPdKeyBytes;
    static constexpr int kState = 8 * NR * kPdPitch * 4 + 64 * NR;          // a warp's state: O, maxima, sums
    static constexpr int kJoined = 8 * NR * 128 * 4 + 64 * NR;              // a CTA's
    // the joined state behind warp 0's where that leaves room, else behind the rings
    static constexpr bool kInside = kState + kJoined <= kBytes;
    static constexpr int kOffJoined = kInside ? kState : kPdWarps * kBytes;
    // queries behind the rings (their place is the joined state's at the end): fp16, or two
    // bf16 terms
    static constexpr int kTerms = kPack ? 1 : 2, kQ = NR * kTerms * 2048;
    static constexpr bool kQRegs = kPack && NR == 1;    // every warp keeps them in registers
    static constexpr int kSmem = kPdWarps * kBytes + (kInside || kQ > kJoined ? kQ : kJoined);
    static_assert(kState <= kBytes, "states over the rings");
    static_assert(kCtas * (kSmem + 1024) <= 228 * 1024, "shared memory of an SM");
};

// The running maximum of a row that has seen no key: any score is above it.
constexpr float kNothing = -3.4028234e38f;

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

// d = a b + c in fp16, c the same in every row
__device__ __forceinline__ void mma_f16_from(float *d, const uint32_t *a, uint32_t b0, uint32_t b1, const float *c)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %11, %10, %11};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]));
}

// d += a b in fp16
__device__ __forceinline__ void mma_f16(float *d, const uint32_t *a, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack2_f16(float lo, float hi)
{
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float2 unpack2_f16(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }

// x and y as two bf16 terms each
__device__ __forceinline__ void two_terms(float x, float y, uint32_t &hi, uint32_t &lo)
{
    hi = pack2(x, y);
    lo = pack2(x - bf_lo(hi), y - bf_hi(hi));
}

// The 8x8 matrix of a warp's bf16 pairs, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// The tiles that some query of a request meets: packed ones of 32 rows, then bf16
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
};

}  // namespace

// NR: octets of query rows (a call's largest request decides).  kPack: the call has
// packed rows.
template <int NR, bool kPack>
__global__ void __launch_bounds__(kPdThreads, (Ring<NR, kPack>::kCtas))
    k_page_decode(const __grid_constant__ PageArgs a, const __grid_constant__ PageTable t, int n_ctas)
{
    using R = Ring<NR, kPack>;
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
    const uint32_t ring = dec_smem_u32(pd_smem) + (uint32_t)(warp * R::kBytes);
    const bool one_page = a.g.rows % kPdKeys == 0;   // a tile's rows are in one page

    const int n_p = kPack ? tl.n[0] + tl.n[1] : 0;
    auto issue_packed = [&](int i, int stage) {
        if (i < n_p) {
            const int r0 = (i < tl.n[0] ? tl.t0[0] + i : tl.t0[1] + i - tl.n[0]) * kPdPacked;
            const uint32_t dst = ring + (uint32_t)(stage * kPackBytes + 16 * lane);
            const uint8_t *src = a.g.packed + packed_block(a, rq, ids, u, r0) + 16 * lane;
#pragma unroll
            for (int x = 0; x < kPackBytes / 512; ++x)
                copy16(dst + 512 * x, src + 512 * x, true);
        }
        copies_end();
    };
    auto issue = [&](int i, int stage) {
        if (i < n_t) {
            const int r0 = (i < n_p + tl.n[2] ? tl.t0[2] + i - n_p : tl.t0[3] + i - n_p - tl.n[2]) * kPdKeys;
            const uint32_t dst = ring + (uint32_t)(stage * kPdKeyBytes);
            const int ch = lane & 15;
            int64_t base = 0;
            if (one_page) {
                const int pg = page_of(a, r0);
                base = (int64_t)page_id(rq, ids, pg) * a.g.s_page + unit + (int64_t)(r0 - pg * a.g.rows) * 128;
            }
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const int r = (lane >> 4) + 2 * x, j = r0 + r;
                const bool there = tl.seen(j);
                int64_t at = base + r * 128;
                if (!one_page && there) {
                    const int pg = page_of(a, j);
                    at = (int64_t)page_id(rq, ids, pg) * a.g.s_page + unit + (int64_t)(j - pg * a.g.rows) * 128;
                }
                at = there ? at + 8 * ch : 0;
                copy16(dst + (uint32_t)(r * 256 + ((ch ^ ((r & 1) << 2)) << 4)), gk + at, there);
                copy16(dst + (uint32_t)(4096 + r * 256 + ((ch ^ (r & 7)) << 4)), gv + at, there);
            }
        }
        copies_end();
    };
    int it = (int)rank * kPdWarps + warp;
    if constexpr (kPack) {
#pragma unroll
        for (int k = 0; k < R::kPackStages; ++k)
            issue_packed(it + k * step, k);
    } else {
#pragma unroll
        for (int k = 0; k < R::kKeyStages; ++k)
            issue(it + k * step, k);
    }

    // Q^T as the B operand: of row 8 x + n and group g the dims 32 g + 8 c + 0..7, turned by the
    // row's position, pair m in word m of what lane 4 n + c reads.  A warp turns a quarter:
    // dims 4 y .. of the groups gp and gp + 2.
    const uint32_t q_base = dec_smem_u32(pd_smem) + (uint32_t)(kPdWarps * R::kBytes);
    auto q_at = [&](int x, int term, int g) { return q_base + (uint32_t)(((x * R::kTerms + term) * 4 + g) * 512 + 16 * lane); };
    float rs[NR][2];         // what scores of the rows 8 x + 2 c and + 1 are scaled by
    {
        const int gp = warp & 1, y = warp >> 1;
        const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) +
                                 (((int64_t)l * a.total_q + rq.q_off) * a.n_q_heads + h * G) * 128 + 32 * gp + 8 * c + 4 * y;
        float f[NR][2][4];
#pragma unroll
        for (int x = 0; x < NR; ++x) {
            const int r = n + 8 * x, tok = r / G;
            const bool some = r < rows;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint2 v = some ? *reinterpret_cast<const uint2 *>(q + ((int64_t)tok * a.n_q_heads + (r - tok * G)) * 128 + 64 * k)
                                     : make_uint2(0, 0);
                f[x][k][0] = bf_lo(v.x);
                f[x][k][1] = bf_hi(v.x);
                f[x][k][2] = bf_lo(v.y);
                f[x][k][3] = bf_hi(v.y);
            }
            auto turn = [](float &p, float &q2, float2 cs) {
                const float v = fmaf(p, cs.x, -(q2 * cs.y));
                q2 = fmaf(p, cs.y, q2 * cs.x);
                p = v;
            };
            if (some) {
                const int pos = rq.pos0 + tok;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (a.interleaved)   // pairs e & 1 of either group
                        turn(f[x][e >> 1][2 * (e & 1)], f[x][e >> 1][2 * (e & 1) + 1],
                             rope_cs(a.rope, 64, pos, 16 * (gp + 2 * (e >> 1)) + 4 * c + 2 * y + (e & 1)));
                    else
                        turn(f[x][0][e], f[x][1][e], rope_cs(a.rope, 64, pos, 32 * gp + 8 * c + 4 * y + e));
                }
            }
        }
        if constexpr (kPack) {
            // the rows' largest elements, over the lanes' quads and the warps
            float *tops = reinterpret_cast<float *>(pd_smem + kPdWarps * R::kBytes);   // [row][warp]
#pragma unroll
            for (int x = 0; x < NR; ++x) {
                float top = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    top = fmaxf(top, fmaxf(fabsf(f[x][0][e]), fabsf(f[x][1][e])));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                if (c == 0)
                    tops[4 * (8 * x + n) + warp] = top;
            }
            __syncthreads();
            // 2^k times the largest is in [2^12, 2^13); a row of less than 2^-88 is taken times 2^100, as 2^-k
            // times the scale has to be a number
            auto power = [&](int row) -> int {
                const float4 v = *reinterpret_cast<const float4 *>(tops + 4 * row);
                return min(100, 12 + 127 - (int)(__float_as_uint(fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w))) >> 23));
            };
            float up[NR];
#pragma unroll
            for (int x = 0; x < NR; ++x) {
                up[x] = __uint_as_float((uint32_t)(127 + power(8 * x + n)) << 23);
#pragma unroll
                for (int e = 0; e < 2; ++e)   // (never 0, which would make the -inf of a hidden row's score a NaN)
                    rs[x][e] = fmaxf(a.scale_log2 * __uint_as_float((uint32_t)(127 - power(8 * x + 2 * c + e)) << 23), 1.40129846e-45f);
            }
            __syncthreads();
#pragma unroll
            for (int x = 0; x < NR; ++x)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    // (the pairs that meet the nibbles four bits higher are a sixteenth)
                    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(q_at(x, 0, gp + 2 * k) + 8u * (uint32_t)y),
                                 "r"(pack2_f16(f[x][k][0] * up[x], f[x][k][1] * up[x])),
                                 "r"(pack2_f16(f[x][k][2] * up[x] * 0.0625f, f[x][k][3] * up[x] * 0.0625f))
                                 : "memory");
        } else {
#pragma unroll
            for (int x = 0; x < NR; ++x) {
                rs[x][0] = rs[x][1] = a.scale_log2;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint32_t hi[2], lo[2];
                    two_terms(f[x][k][0], f[x][k][1], hi[0], lo[0]);
                    two_terms(f[x][k][2], f[x][k][3], hi[1], lo[1]);
                    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(q_at(x, 0, gp + 2 * k) + 8u * (uint32_t)y), "r"(hi[0]), "r"(hi[1]) : "memory");
                    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(q_at(x, 1, gp + 2 * k) + 8u * (uint32_t)y), "r"(lo[0]), "r"(lo[1]) : "memory");
                }
            }
        }
        __syncthreads();
    }
    uint4 qr[R::kQRegs ? 4 : 1];
    if constexpr (R::kQRegs) {
#pragma unroll
        for (int g = 0; g < 4; ++g)
            qr[g] = lds128(q_at(0, 0, g));
    }
    auto query = [&](int x, int term, int g) -> uint4 {
        if constexpr (R::kQRegs)
            return qr[g];
        else
            return lds128(q_at(x, term, g));
    };
    float start[kPack ? NR : 1][4][2];   // -8 times a group's sum, of rows 8 x + 2 c and + 1
    if constexpr (kPack) {
#pragma unroll
        for (int x = 0; x < NR; ++x)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const uint4 q = query(x, 0, g);
                const float2 v[4] = {unpack2_f16(q.x), unpack2_f16(q.y), unpack2_f16(q.z), unpack2_f16(q.w)};
                float s = fmaf(16.f, (v[1].x + v[1].y) + (v[3].x + v[3].y), (v[0].x + v[0].y) + (v[2].x + v[2].y));
                s += __shfl_xor_sync(0xffffffffu, s, 1);
                s += __shfl_xor_sync(0xffffffffu, s, 2);
                s *= -8.f / 16777216.f;
                start[x][g][0] = __shfl_sync(0xffffffffu, s, 8 * c);
                start[x][g][1] = __shfl_sync(0xffffffffu, s, 8 * c + 4);
            }
    }
    // rows that every query sees: below, and from (or among the first) on
    const int all_hi = min(rq.kv_len, rq.pos0 + 1), all_lo = a.window > 0 ? rq.pos0 + rq.q_len - a.window : 0;

    float m_run[NR][2], l_run[NR][2];   // of query rows 8 x + 2 c and + 1; l over this lane's keys
    float o[NR][8][4];                  // dims 16 j + n and + 8 of these two rows
#pragma unroll
    for (int x = 0; x < NR; ++x) {
        m_run[x][0] = m_run[x][1] = kNothing;
        l_run[x][0] = l_run[x][1] = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            o[x][j][0] = o[x][j][1] = o[x][j][2] = o[x][j][3] = 0.f;
    }

    // One step: 16 rows from `row` on, packed at `st` (kThin) or as bf16 rows.  `all`: every
    // query sees every row.
    auto step16 = [&](auto thin, int row, uint32_t st, bool all) {
        constexpr bool kThin = decltype(thin)::value;
        const uint32_t kb = st + 16 * lane, sb = st + 1024 + 16 * n;
        // S^T: keys n and n + 8 of the 16, query rows 8 x + 2 c and + 1
        float s[NR][4];
#pragma unroll
        for (int x = 0; x < NR; ++x)
            s[x][0] = s[x][1] = s[x][2] = s[x][3] = 0.f;
        if constexpr (kThin) {
            const uint4 c0 = lds128(kb), c1 = lds128(kb + 512);
            const uint4 z = lds128(sb);
            const uint32_t w0[4] = {c0.x, c0.y, c0.z, c0.w}, w1[4] = {c1.x, c1.y, c1.z, c1.w};
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const uint32_t y0 = g < 2 ? z.x : z.y, y1 = g < 2 ? z.z : z.w;
                const float x0 = (g & 1) ? bf_hi(y0) : bf_lo(y0), x1 = (g & 1) ? bf_hi(y1) : bf_lo(y1);
                // pairs 0 and 2 of the words; pairs 1 and 3, which are 16 times as much
                const uint32_t v0 = w0[g] >> 8, v1 = w1[g] >> 8;
                const uint32_t a0[4] = {w0[g] & 0x000f000fu, w1[g] & 0x000f000fu, v0 & 0x000f000fu, v1 & 0x000f000fu};
                const uint32_t a1[4] = {w0[g] & 0x00f000f0u, w1[g] & 0x00f000f0u, v0 & 0x00f000f0u, v1 & 0x00f000f0u};
#pragma unroll
                for (int x = 0; x < NR; ++x) {
                    const uint4 q = query(x, 0, g);
                    float d[4];
                    mma_f16_from(d, a0, q.x, q.z, start[x][g]);
                    mma_f16(d, a1, q.y, q.w);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[x][e] = fmaf(e < 2 ? x0 : x1, d[e], s[x][e]);
                }
            }
        } else {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const uint32_t at = st + (uint32_t)(n * 256 + (((4 * g + c) ^ ((n & 1) << 2)) << 4));
                const uint4 w0 = lds128(at), w1 = lds128(at + 2048);
                const uint32_t a0[4] = {w0.x, w1.x, w0.y, w1.y}, a1[4] = {w0.z, w1.z, w0.w, w1.w};
#pragma unroll
                for (int x = 0; x < NR; ++x) {
                    uint32_t hi[4], lo[4];
                    if constexpr (kPack) {   // (the few rows behind the packed ones: exactly, 8 and 3 bits)
                        const uint4 q = query(x, 0, g);
                        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            const float2 v = unpack2_f16(w[m]);
                            two_terms(v.x * ((m & 1) ? 16.f : 1.f), v.y * ((m & 1) ? 16.f : 1.f), hi[m], lo[m]);
                        }
                    } else {
                        const uint4 p = query(x, 0, g), q = query(x, 1, g);
                        hi[0] = p.x, hi[1] = p.y, hi[2] = p.z, hi[3] = p.w;
                        lo[0] = q.x, lo[1] = q.y, lo[2] = q.z, lo[3] = q.w;
                    }
                    mma_bf16(s[x], a0, lo[0], lo[1]);
                    mma_bf16(s[x], a1, lo[2], lo[3]);
                    mma_bf16(s[x], a0, hi[0], hi[1]);
                    mma_bf16(s[x], a1, hi[2], hi[3]);
                }
            }
        }
        if (!all) {
#pragma unroll
            for (int x = 0; x < NR; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const Sees see = sees(a, rq, min(rq.pos0 + rq.q_len - 1, rq.pos0 + (8 * x + 2 * c + (e & 1)) / G));
                    if (!see(row + n + 8 * (e >> 1)))
                        s[x][e] = -INFINITY;
                }
        }
        // Scores become probabilities relative to the row's maximum, which moves only when a
        // score is more than 8 (log2) above it: bf16 and fp32 hold that, and most steps need
        // no exchange between the lanes.
        constexpr float kUnit = kThin ? 16777216.f : 1.f;   // (packed keys' scores are in 2^-24)
        float t[NR][4];
        float over = -INFINITY;
#pragma unroll
        for (int x = 0; x < NR; ++x) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                t[x][e] = fmaf(s[x][e], rs[x][e & 1] * kUnit, -m_run[x][e & 1]);
            over = fmaxf(over, fmaxf(fmaxf(t[x][0], t[x][1]), fmaxf(t[x][2], t[x][3])));
        }
        if (__any_sync(0xffffffffu, over > 8.f)) {
#pragma unroll
            for (int x = 0; x < NR; ++x)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float sc = rs[x][e] * kUnit;
                    float mx = fmaxf(s[x][e], s[x][e + 2]) * sc;
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                    mx = fmaxf(mx, m_run[x][e]);
                    const float corr = dec_ex2(m_run[x][e] - mx);
                    m_run[x][e] = mx;
                    l_run[x][e] *= corr;
                    t[x][e] = fmaf(s[x][e], sc, -mx);
                    t[x][e + 2] = fmaf(s[x][e + 2], sc, -mx);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        o[x][j][e] *= corr;
                        o[x][j][e + 2] *= corr;
                    }
                }
        }
#pragma unroll
        for (int x = 0; x < NR; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                t[x][e] = dec_ex2(t[x][e]);
                l_run[x][e & 1] += t[x][e];
            }
        // O^T += V^T P^T
        if constexpr (kThin) {
            const uint4 c0 = lds128(kb + kPackPart), c1 = lds128(kb + kPackPart + 512);
            uint4 z = lds128(sb + kPackPart);
            if (!all) {   // rows that no query sees may have scales of NaN
                if (!tl.seen(row + n))
                    z.x = z.y = 0u;
                if (!tl.seen(row + n + 8))
                    z.z = z.w = 0u;
            }
            const uint32_t w0[4] = {c0.x, c0.y, c0.z, c0.w}, w1[4] = {c1.x, c1.y, c1.z, c1.w};
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const uint32_t y0 = g < 2 ? z.x : z.y, y1 = g < 2 ? z.z : z.w;
                const float x0 = (g & 1) ? bf_hi(y0) : bf_lo(y0), x1 = (g & 1) ? bf_hi(y1) : bf_lo(y1);
                uint32_t b0[NR], b1[NR];
#pragma unroll
                for (int x = 0; x < NR; ++x) {
                    b0[x] = transpose8(pack2(t[x][0] * x0, t[x][1] * x0));
                    b1[x] = transpose8(pack2(t[x][2] * x1, t[x][3] * x1));
                }
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const uint32_t va[4] = {less136(pair128(w0[g] >> (8 * m))), less136(pair128(w0[g] >> (8 * m + 4))),
                                            less136(pair128(w1[g] >> (8 * m))), less136(pair128(w1[g] >> (8 * m + 4)))};
#pragma unroll
                    for (int x = 0; x < NR; ++x)
                        mma_bf16(o[x][2 * g + m], va, b0[x], b1[x]);
                }
            }
        } else {
            uint32_t b0[NR][2], b1[NR][2];   // two terms
#pragma unroll
            for (int x = 0; x < NR; ++x) {
                two_terms(t[x][0], t[x][1], b0[x][0], b0[x][1]);
                two_terms(t[x][2], t[x][3], b1[x][0], b1[x][1]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    b0[x][e] = transpose8(b0[x][e]);
                    b1[x][e] = transpose8(b1[x][e]);
                }
            }
            const int key = (lane & 7) + 8 * (lane >> 4);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint32_t va[4];
                ldsm_x4_t(st + (uint32_t)(4096 + key * 256 + (((2 * j + ((lane >> 3) & 1)) ^ (key & 7)) << 4)), va[0], va[1], va[2], va[3]);
#pragma unroll
                for (int x = 0; x < NR; ++x) {
                    mma_bf16(o[x][j], va, b0[x][1], b1[x][1]);
                    mma_bf16(o[x][j], va, b0[x][0], b1[x][0]);
                }
            }
        }
    };
    auto all_see = [&](int row, int end) { return end <= all_hi && (row >= all_lo || end <= a.n_first); };
    if constexpr (kPack) {
        for (int stage = 0; it < n_p; it += step, stage = stage + 1 == R::kPackStages ? 0 : stage + 1) {
            copies_wait<R::kPackStages - 1>();
            __syncwarp();
            const int row0 = (it < tl.n[0] ? tl.t0[0] + it : tl.t0[1] + it - tl.n[0]) * kPdPacked;
            const bool all = all_see(row0, row0 + kPdPacked);
            // (a loop, which the instruction cache holds)
#pragma unroll 1
            for (int k = 0; k < kPdPacked / kPdKeys; ++k)
                step16(std::true_type(), row0 + kPdKeys * k, ring + (uint32_t)(stage * kPackBytes + k * kPackStep), all);
            __syncwarp();
            issue_packed(it + R::kPackStages * step, stage);
        }
        issue(it, 0);   // (the ring is free: what was in flight behind the last tile is nothing)
    }
    for (int stage = 0; it < n_t; it += step, stage = stage + 1 == R::kKeyStages ? 0 : stage + 1) {
        copies_wait<R::kKeyStages - 1>();
        __syncwarp();
        const int row0 = (it < n_p + tl.n[2] ? tl.t0[2] + it - n_p : tl.t0[3] + it - n_p - tl.n[2]) * kPdKeys;
        step16(std::false_type(), row0, ring + (uint32_t)(stage * kPdKeyBytes), all_see(row0, row0 + kPdKeys));
        __syncwarp();
        issue(it + R::kKeyStages * step, stage);
    }
    copies_wait<0>();
    __syncwarp();

    // the warp's state over its ring
    auto area = [&](int w) { return reinterpret_cast<float *>(pd_smem + w * R::kBytes); };
    {
        float *f = area(warp);
#pragma unroll
        for (int x = 0; x < NR; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * x + 2 * c + e;
                float v = l_run[x][e];
                v += __shfl_xor_sync(0xffffffffu, v, 4);
                v += __shfl_xor_sync(0xffffffffu, v, 8);
                v += __shfl_xor_sync(0xffffffffu, v, 16);
                if (n == 0) {
                    f[8 * NR * kPdPitch + r] = m_run[x][e];
                    f[8 * NR * kPdPitch + 8 * NR + r] = v;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    f[r * kPdPitch + 16 * j + n] = o[x][j][e];
                    f[r * kPdPitch + 16 * j + n + 8] = o[x][j][e + 2];
                }
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
    float *joined = reinterpret_cast<float *>(pd_smem + R::kOffJoined);   // [8 NR][128], maxima, sums
    for (int r = warp; r < rows; r += kPdWarps) {
        float M = kNothing, L = 0.f;
#pragma unroll
        for (int w = 0; w < kPdWarps; ++w)
            M = fmaxf(M, area(w)[8 * NR * kPdPitch + r]);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kPdWarps; ++w) {
            const float f = dec_ex2(area(w)[8 * NR * kPdPitch + r] - M);
            const float4 x = *reinterpret_cast<const float4 *>(area(w) + r * kPdPitch + col);
            L = fmaf(area(w)[8 * NR * kPdPitch + 8 * NR + r], f, L);
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
                joined[8 * NR * 128 + r] = M;
                joined[8 * NR * 128 + 8 * NR + r] = L;
            }
        }
    }
    if (n_ctas == 1)
        return;
    cluster_meet();
    const uint32_t mine = dec_smem_u32(joined);
    for (int r = (int)rank + n_ctas * warp; r < rows; r += n_ctas * kPdWarps) {
        float M = kNothing, L = 0.f;
        for (int k = 0; k < n_ctas; ++k)
            M = fmaxf(M, ld_cluster1(at_rank(mine + 4u * (uint32_t)(8 * NR * 128 + r), (uint32_t)k)));
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < n_ctas; ++k) {
            const float mk = ld_cluster1(at_rank(mine + 4u * (uint32_t)(8 * NR * 128 + r), (uint32_t)k));
            const float lk = ld_cluster1(at_rank(mine + 4u * (uint32_t)(8 * NR * 128 + 8 * NR + r), (uint32_t)k));
            const float4 x = ld_cluster(at_rank(mine + 4u * (uint32_t)(r * 128 + col), (uint32_t)k));
            const float f = dec_ex2(mk - M);
            L = fmaf(lk, f, L);
            v.x = fmaf(x.x, f, v.x);
            v.y = fmaf(x.y, f, v.y);
            v.z = fmaf(x.z, f, v.z);
            v.w = fmaf(x.w, f, v.w);
        }
        write(r, col, M, L, v);
    }
    cluster_meet();   // a CTA's state is read by the others until here
}

namespace {

struct Variant {
    void (*kernel)(PageArgs, PageTable, int);
    int smem, ctas;
};
template <int NR, bool kPack>
Variant variant()
{
    return {k_page_decode<NR, kPack>, Ring<NR, kPack>::kSmem, Ring<NR, kPack>::kCtas};
}

// Clusters of 1, 2, 4 and 8 CTAs that the device holds at once.
cudaError_t capacities(const Variant &v, int (&cap)[4])
{
    cudaError_t e = cudaFuncSetAttribute(v.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, v.smem);
    for (int i = 0; i < 4 && e == cudaSuccess; ++i) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(8u << i);
        cfg.blockDim = dim3(kPdThreads);
        cfg.dynamicSmemBytes = (size_t)v.smem;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 1u << i;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&cap[i], v.kernel, &cfg);
    }
    return e;
}

}  // namespace

cudaError_t launch_page_decode(const PageArgs &a, const PageTable &t, const DevPageReq *host_reqs, int n_sms, cudaStream_t s)
{
    const Variant variants[4] = {variant<1, false>(), variant<2, false>(), variant<1, true>(), variant<2, true>()};
    static std::atomic<bool> known[64] = {};   // per device (host threads may race: same values)
    static std::atomic<int> caps[64][4][4];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    int cap[4][4];
    if (dev < 64 && known[dev].load(std::memory_order_acquire)) {
        for (int i = 0; i < 16; ++i)
            cap[i / 4][i % 4] = caps[dev][i / 4][i % 4].load(std::memory_order_relaxed);
    } else {
        for (int i = 0; i < 4; ++i)
            if ((e = capacities(variants[i], cap[i])) != cudaSuccess)
                return e;
        if (dev < 64) {
            for (int i = 0; i < 16; ++i)
                caps[dev][i / 4][i % 4].store(cap[i / 4][i % 4], std::memory_order_relaxed);
            known[dev].store(true, std::memory_order_release);
        }
    }
    const int units = a.n_layers * a.n_kv_heads, G = a.n_q_heads / a.n_kv_heads;
    int64_t few = 0, bytes = 0;   // of one unit's tiles
    int rows = 0;
    bool packed = false;
    for (int b = 0; b < a.n_reqs; ++b) {
        const int64_t r = host_reqs[b].q_len * (int64_t)G;
        if (r == 0 || r > kPageFewRows)
            continue;
        TileList tl;
        tl.set(host_reqs[b], a.window, a.n_first);
        bytes += (int64_t)(tl.n[0] + tl.n[1]) * kPackBytes + (int64_t)(tl.n[2] + tl.n[3]) * kPdKeyBytes;
        packed = packed || tl.n[0] + tl.n[1] > 0;
        rows = std::max(rows, (int)r);
        ++few;
    }
    if (few == 0)
        return cudaSuccess;
    const int which = (packed ? 2 : 0) + (rows > 8 ? 1 : 0);
    // CTAs of a (request, unit), by an estimate of the call's time in us: 6 to start and end;
    // the bytes at the card's pace (6.4 TB/s, on packed rows at the instructions', 4.1); where all
    // clusters are resident at once the fullest SM's share at that SM's pace (36, 54, 60
    // GB/s for one, two, three CTAs; 19 and 27 packed); else 5 for each round behind the
    // first and half a CTA's time for the last ones.  Measured with 1, 2, 4, 8 CTAs:
    //   bf16, 2,656 rows: 112 units 45, 31, 42, 44 us; 32 units 43, 26, 17, 15; 336
    //     (request, unit) pairs 72, 80, 88, 103; 4,100 rows, 256 units: 90, 115, 98, 113
    //   packed, 33,280 rows: 256 units 355, 320, 301, 288 us; 16 units 255, 136, 75, 50;
    //     1,216 rows, 288 units 20, 20, 25, 38
    const double pace[2][3] = {{36e3, 54e3, 60e3}, {19e3, 27e3, 27e3}}, total = (double)bytes * units;
    int c = 1;
    double best = 1e30;
    for (int i = 0; i < 4; ++i) {
        const int64_t n = few * units << i, room = std::max<int64_t>(1, (int64_t)cap[which][i] << i);
        const double cta = (double)bytes / (double)(few << i);   // bytes of one
        double us = total / (packed ? 4.1e6 : 6.4e6);
        if (n <= room) {
            const int64_t k = (n + n_sms - 1) / n_sms;
            us = std::max(us, (double)k * cta / pace[packed][std::min<int64_t>(k, 3) - 1]);
        } else {
            us += 5. * (double)((n - 1) / room) + 0.5 * cta / pace[packed][0];
        }
        us += i ? 1. : 0.;
        if (us < 0.97 * best) {
            best = us;
            c = 1 << i;
        }
    }
    const Variant &v = variants[which];
    return launch_cluster(v.kernel, (int64_t)a.n_reqs * units * c, kPdThreads, v.smem, c, s, a, t, c);
}

}  // namespace kvr
