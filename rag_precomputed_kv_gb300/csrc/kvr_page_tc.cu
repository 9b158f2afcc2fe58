// kvr_page_tc.cu -- attention of many query rows over a paged cache, on the
// tensor cores (bf16, head_dim 128).
//
// The G query heads of a kv head are packed into the rows (row = token * G + g), as
// in the query prefill; a request's rows of one (layer, kv-head) meet its cache in
// blocks of up to 256, two 128-row tiles A and B per CTA with S, P and O in TMEM.
// The key tiles of a block are 128 rows each of a list: the first rows and the window's that its
// queries see, rounded out to TMA boxes (4 first rows and a window of 1,024 are 9 tiles for 64 tokens;
// with tiles aligned in the cache 10).
//
//   warps 0-3, 4-7  softmax of tile A, B, a row a thread, and its output;
//   warp 8          works out each item's block of rows and its tiles, and passes them to
//                   the others through a ring of three, then loads by TMA: a tile's
//                   pages are boxes of 16 to 128 rows, one and a panel a lane (small ones
//                   together with warp 10);
//   warp 9          tcgen05 products; rows of V that no query of the request sees become
//                   zeros first (their weight is 0, but 0 x NaN is NaN);
//   warps 10, 11    else tiles of pages that TMA boxes cannot bring (their rows are no multiple
//                   of 16 or lie at odd strides), 64 rows each.
// A slot's barrier counts two arrivals whichever way it is filled: two of warp 8, or
// one each of warps 10 and 11.  That a slot is free for them, warps 10 and 11 learn from
// warp 8, over a barrier of the slot that completes a phase for each of their tiles and
// no other: on the barrier that frees slots they could come two phases late, past tiles
// that are none of theirs, and a wait for a parity would not return.
//
// Packed rows are restored to bf16 first (k_page_restore: scale * code, rounded), slice by
// slice of the (layer, kv-head) units as the scratch holds them, once for all blocks of a
// request.  (8 x 64 tokens x 7 heads on 2,592 packed rows, 112 units: restored by warps 10
// and 11 on the way instead, for every block again, a step of 128 keys took 8.8 us and the
// call 2,140; with k_page_restore 820 at once, 735 now.)
//
// Few blocks (fewer than the SMs): each is cut in stretches of key tiles, whose
// partial results (O relative to a maximum, the maximum, the sum) k_page_join adds.
// Rounded to bf16 on the way: the turned queries, the probabilities, and what packed
// rows stand for (all operands of products with bf16 numbers; 0.0025 to 0.0036 of the
// output's norm, its own rounding 0.0017 of it.  A second term of the queries or the
// probabilities would add half of all products).
//
// Bound by the tensor pipe and the chain S, softmax, P V of each tile: a step of 128 keys and
// 256 rows takes 1.5 us, its products 1.35 at cuBLAS's rate.  A 4,096-token prompt x 4 heads, 64 units, 880 to 889 us without a window, 0.64 of
// the measured peak; 256 units with a window of 1,024 and 64 first rows (9 key tiles a block) 1,965 to
// 2,030 us, where 5 of a block's 18 us are its start and end.  What mattered (that prompt): registers without
// spills (28 bytes spilled in the softmax: 8 %), masks as bits, item geometry and page numbers
// worked out ahead of their use, the next item's S ahead of the epilogue (2,460 then); 64 bytes
// written at once by lanes in pairs (a row a thread: 12 bytes a clock; 4 %); one tile for first rows and
// window (9 %); little code in an item's start and end, by loops (7 %: rescale, masks and output are
// executed once a block, and their code has to come from far); V waited for before the probabilities,
// queries of either tile on a barrier of their own.  Not kept: the next item's S between the last two
// products (its softmax then runs beside the other tile's output, 10 % slower), the next geometry
// behind the queries' load (8 %).
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "kvr_page_common.cuh"
#include "kvr_tc_common.cuh"

namespace kvr {

namespace {

using namespace page;
using namespace tc;

constexpr int kPtThreads = 384;
constexpr int kPtRegsLaunch = 168, kPtRegsSoftmax = 208, kPtRegsOther = 88;
static_assert(2 * 128 * kPtRegsSoftmax + 128 * kPtRegsOther <= kPtThreads * kPtRegsLaunch, "register split");
constexpr int kPtTile = 128;                        // keys per tile, rows per query tile
constexpr int kPtSlots = 5;                         // K/V ring
constexpr int kPtGeos = 3;                          // geometry ring
constexpr int kPtTileBytes = kPtTile * 128 * 2;     // 32 KB
constexpr int kPtPanel = kPtTileBytes / 2;
constexpr int kPtTmemCols = 512;
__host__ __device__ constexpr uint32_t pt_col_s(int x) { return 128u * (uint32_t)x; }
__host__ __device__ constexpr uint32_t pt_col_o(int x) { return 256u + 128u * (uint32_t)x; }
constexpr float kPtRescale = 8.0f;

constexpr int kPtOffQ = 0;
constexpr int kPtOffKV = 2 * kPtTileBytes;
constexpr int kPtOffBar = kPtOffKV + kPtSlots * kPtTileBytes;
constexpr int kTbFull = 0, kTbEmpty = kTbFull + kPtSlots, kTbS = kTbEmpty + kPtSlots, kTbP = kTbS + 2, kTbO = kTbP + 2,
              kTbOEmpty = kTbO + 2, kTbPv = kTbOEmpty + 2, kTbQ = kTbPv + 1, kTbQEmpty = kTbQ + 2, kTbDrain = kTbQEmpty + 1,
              kTbJob = kTbDrain + 1, kTbGeo = kTbJob + kPtSlots, kTbGeoFree = kTbGeo + kPtGeos, kTbNum = kTbGeoFree + kPtGeos;
constexpr int kPtOffMisc = kPtOffBar + 8 * kTbNum;
constexpr int kPtOffGeo = (kPtOffMisc + 16 + 15) & ~15;
constexpr int kPtGeoBytes = 160;
constexpr int kPtSmem = kPtOffGeo + kPtGeos * kPtGeoBytes + 1024;     // + alignment slack
static_assert(kPtSmem <= 227 * 1024, "shared memory budget");

constexpr uint32_t kPtIdescS = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kPtTile >> 3) << 17) |
                               ((uint32_t)(kPtTile >> 4) << 24);
constexpr uint32_t kPtIdescPV = kPtIdescS | (1u << 16);   // V is MN-major

// A partial result: per tile x, O as float4 [column / 4][row] (lanes are rows:
// coalesced), then (max, sum) [row].
constexpr int64_t kPartO = 2 * 128 * 128;                        // floats
constexpr int64_t kPartFloats = kPartO + 2 * 128 * 2;
static_assert(kPartFloats * 4 == kPagePartBytes, "partial result layout");
__device__ __forceinline__ float4 *part_o(float *part, int64_t slot, int x)
{
    return reinterpret_cast<float4 *>(part + slot * kPartFloats) + x * (128 * 32);
}
__device__ __forceinline__ float2 *part_ml(float *part, int64_t slot, int x)
{
    return reinterpret_cast<float2 *>(part + slot * kPartFloats + kPartO) + x * 128;
}

// One block of query rows, and the key tiles of it that an item takes.
struct alignas(16) Block {
    DevPageReq rq;
    int lh, l, h;
    int row0, rows, nx;      // first packed row in the request, rows (<= 256), 128-row tiles
    int hi, lo;              // rows that some query of the block sees: j < hi and (j >= lo or a first one)
    Sees any;                // ... and of the request
    int all_hi, all_lo;      // rows that all its queries see: j < all_hi and (j >= all_lo or a first one)
    int first, shift;        // place v of the list of rows is row v, from `first` on row v + shift
    int jb, je;              // the item's 128-row tiles of the list

    int rest_first, rest_row[2];   // row j is restored row rest_row[j >= rest_first] + j
    int64_t unit;            // elements from a page's start to the (layer, kv-head)'s first row

    __device__ __forceinline__ int row(int v) const { return v < first ? v : v + shift; }
    // tile j has first rows and others
    __device__ __forceinline__ bool cut(int j) const { return shift > 0 && j * kPtTile < first && j * kPtTile + kPtTile > first; }
    __device__ __forceinline__ bool all_seen(int j0, int j1) const { return j1 <= any.hi && (j0 >= any.lo || j1 <= any.few); }
    __device__ __forceinline__ bool some_seen(int j0, int j1) const { return j0 < any.few || (j0 < any.hi && j1 > any.lo); }
    // tile j is one of restored rows (a request's that has packed ones are whole tiles of its cache)
    __device__ __forceinline__ bool restored(int j) const { return rq.packed_len > 0 && row(j * kPtTile) < rq.packed_len; }
    __device__ __forceinline__ int place(int j) const { return j + (j < rest_first ? rest_row[0] : rest_row[1]); }
};
static_assert(sizeof(Block) <= kPtGeoBytes, "geometry ring");

__device__ __forceinline__ Block block_at(const PageArgs &a, const PageTcArgs &p, const DevPageReq *reqs, int64_t w)
{
    Block s;
    const int lh_s = (int)(w / p.unit_items), in_unit = (int)(w - (int64_t)lh_s * p.unit_items);
    s.lh = p.lh_base + lh_s;
    int lo = 0, hi = a.n_reqs - 1;
    while (lo < hi) {   // the last request whose first item is <= it (one with items)
        const int mid = (lo + hi + 1) >> 1;
        if (reqs[mid].item0 <= in_unit)
            lo = mid;
        else
            hi = mid - 1;
    }
    s.rq = reqs[lo];
    s.l = s.lh / a.n_kv_heads;
    s.h = s.lh - s.l * a.n_kv_heads;
    s.unit = s.l * a.g.s_layer + s.h * a.g.s_head;
    const int G = a.n_q_heads / a.n_kv_heads, all = s.rq.q_len * G, mb = (all + 255) >> 8;
    const int i = in_unit - s.rq.item0, blk = mb - 1 - i / p.splits, sp = i % p.splits;   // (the last blocks see most: first)
    s.row0 = blk * 256;
    s.rows = min(256, all - s.row0);
    s.nx = s.rows > 128 ? 2 : 1;
    const int p0 = s.rq.pos0 + s.row0 / G, p1 = s.rq.pos0 + (s.row0 + s.rows - 1) / G;   // its first and last token
    s.hi = min(s.rq.kv_len, p1 + 1);
    s.lo = min(s.hi, a.window > 0 ? max(0, p0 - a.window + 1) : 0);
    s.all_hi = min(s.rq.kv_len, p0 + 1);
    s.all_lo = a.window > 0 ? p1 - a.window + 1 : 0;
    s.any = sees_any(a, s.rq);
    const RestTiles rest = rest_tiles(s.any.hi, s.any.lo, s.any.few, s.rq.packed_len);
    s.rest_first = rest.first * kPtTile;
    s.rest_row[0] = (lh_s * p.unit_tiles + s.rq.tile0) * kPtTile;
    s.rest_row[1] = s.rest_row[0] + (rest.first - rest.win) * kPtTile;
    // the rows listed: the first ones and those from s.lo on, both rounded out to whole boxes; 32 places
    // in a row hold rows in a row
    const int g = s.rq.packed_len > 0 ? kPtTile : p.box ? p.box : 16, g32 = max(g, 32);   // (powers of two)
    s.first = (min(a.n_first, s.lo) + g32 - 1) & -g32;
    const int w0 = max(s.first, s.lo & -g);
    s.shift = w0 - s.first;
    const int n = (s.first + (s.lo < s.hi ? max(0, s.hi - w0) : 0) + kPtTile - 1) / kPtTile;
    s.jb = (int)((int64_t)n * sp / p.splits);
    s.je = (int)((int64_t)n * (sp + 1) / p.splits);
    return s;
}

__device__ __forceinline__ void st_global_v8(void *p, const uint32_t (&v)[8])
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                 "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// 16 bytes to shared memory, on the way until the thread waits for its copies; or zeros.
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

constexpr int kLoadOne = 0, kLoadTwo = 1, kLoadByHand = 2;
// A tile that warps 10 and 11 fill.
template <int kLoad>
__device__ __forceinline__ bool by_hand(const Block &s, int j)
{
    return kLoad == kLoadByHand && !s.restored(j);
}

}  // namespace

// kOne: every block of the call has one 128-row tile.  The S of its next key tile then
// goes into tile B's buffer, ahead of the softmax (32 tokens x 4 heads on 33,000 rows, 64
// units: 253 -> 231 us; as a branch of the kernel for two tiles it cost those 10 %).
// kLoad, who brings the pages: warp 8 by TMA; kLoadTwo: warp 10 beside it, a 64-column panel each;
// kLoadByHand: warps 10 and 11 (branches of one kernel for these cost the first 2 %).  A load of 16-
// or 32-row boxes takes one warp longer than a step: 4,096-token prompt, window 1,024, 4 first rows, 64
// units, pages of 16 rows 638 -> 532 us, of 32 540 -> 519; 8 windows of 4,100 rows in pages of 16, 8
// tokens 971 -> 780.  Boxes of 64: the prompt 507, by two warps 518; blocks of one tile gain (185 -> 182).
// By hand three tiles are in flight (pages of 20 rows, 4 x 8 tokens on 2,656 rows, 32 units: 94 us; 946
// with loads that the warps wait for).
template <bool kOne, int kLoad>
__global__ void __launch_bounds__(kPtThreads, 1)
    k_page_attention(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                     const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmrk,
                     const __grid_constant__ CUtensorMap tmrv, const __grid_constant__ PageArgs a,
                     const __grid_constant__ PageTcArgs p, const __grid_constant__ PageTable pt)
{
    extern __shared__ uint8_t pt_smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(pt_smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    auto bar = [&](int i) { return sbase + kPtOffBar + 8u * (uint32_t)i; };
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kPtOffMisc + 4);
    constexpr bool kTwo = kLoad == kLoadTwo;
    const bool second = kTwo && threadIdx.x >> 5 == 10;   // a second warp 8
    const int warp = second ? 8 : (int)(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const DevPageReq *reqs = a.reqs ? a.reqs : pt.reqs;
    const int32_t *ids = a.reqs ? a.ids : pt.ids;
    const int G = a.n_q_heads / a.n_kv_heads;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kTbNum; ++i)
            mbar_init(bar(i), i < kTbEmpty ? 2u
                              : (i >= kTbP && i < kTbP + 2) || (i >= kTbOEmpty && i < kTbOEmpty + 2) ? 4u
                              : i >= kTbGeoFree ? 11u
                                                                                                    : 1u);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 9)
        tmem_alloc(sbase + kPtOffMisc, kPtTmemCols);
    if (warp == 8 && !second && lane == 0) {
        prefetch_tmap(&tmq);
        prefetch_tmap(&tmk);
        prefetch_tmap(&tmv);
        prefetch_tmap(&tmrk);
        prefetch_tmap(&tmrv);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + kPtOffMisc);
    // the CTA's item i: its geometry, once it is there; at last free it for item i + kPtGeos
    auto geo = [&](int i) -> const Block & { return *reinterpret_cast<const Block *>(smem + kPtOffGeo + i % kPtGeos * kPtGeoBytes); };
    auto geo_wait = [&](int i) -> bool {
        return mbar_wait_warp(bar(kTbGeo + i % kPtGeos), (uint32_t)(i / kPtGeos) & 1, abort_flag);
    };
    auto geo_done = [&](int i) {
        __syncwarp();
        if (lane == 0)
            mbar_arrive(bar(kTbGeoFree + i % kPtGeos));
    };
    // one arrival of a warp, behind what its lanes did to TMEM
    auto warp_arrive = [&](int i) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0)
            mbar_arrive(bar(i));
    };
    const int n_items = (int)((p.total - blockIdx.x + gridDim.x - 1) / gridDim.x);

    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPtRegsSoftmax));
        pdl_wait_prerequisites();
        pdl_launch_dependents();
        const int x = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const float sc = a.scale_log2;
        int s_cnt = 0, alt_cnt = 0, o_cnt = 0, pv_cnt = 0;   // phases seen of S, of the second buffer's S, of O, of single P V's
        bool ok = true;
        for (int item = 0; item < n_items; ++item) {
            if (!geo_wait(item)) {
                ok = false;
                break;
            }
            // (read where it is needed: the scores leave few registers)
            const Block &b = geo(item);
            if (x >= b.nx) {
                geo_done(item);
                continue;
            }
            // a warp without rows of its own only keeps the barriers going
            const bool idle = x * 128 + (warp & 3) * 32 >= b.rows;
            const int pos = b.rq.pos0 + (b.row0 + x * 128 + r) / G;
            float m_run = -INFINITY, l_run = 0.f;
            for (int j = b.jb; j < b.je; ++j) {
                const int k0 = b.row(j * kPtTile), k1 = k0 + kPtTile;
                const bool all = !b.cut(j) && k1 <= b.all_hi && (k0 >= b.all_lo || k1 <= a.n_first);
                // (one tile uses both S buffers by turns)
                const bool odd = kOne && ((j - b.jb) & 1);
                const int sb = odd ? 1 : x;
                if (!mbar_wait_warp(bar(kTbS + sb), (uint32_t)(odd ? alt_cnt : s_cnt) & 1u, abort_flag)) {
                    ok = false;
                    break;
                }
                if (odd)
                    ++alt_cnt;
                else
                    ++s_cnt;
                tc_fence_after();
                // (one tile) the P V before is done, O stable: the commit that signalled S does not
                // cover it then, as it does with two tiles
                auto pv_done = [&]() -> bool {
                    if (!kOne || j == b.jb)
                        return true;
                    const bool r = mbar_wait_warp(bar(kTbPv), (uint32_t)pv_cnt & 1u, abort_flag);
                    ++pv_cnt;
                    tc_fence_after();
                    return r;
                };
                if (idle) {
                    ok = pv_done();
                    if (!ok)
                        break;
                    warp_arrive(kTbP + sb);
                    continue;
                }
                const uint32_t s_cols = lane_base + pt_col_s(sb);
                if (!all) {
                    // scores of rows that this query does not see go, in TMEM: a loop over 32 columns (in
                    // place of 128 selects in registers: the code of an item's tiles and its end stays
                    // within what the instruction cache holds)
                    const Sees see = sees(a, b.rq, pos);
                    auto below = [](int n) -> uint32_t {
                        uint32_t r;
                        asm("bmsk.clamp.b32 %0, 0, %1;" : "=r"(r) : "r"(max(n, 0)));
                        return r;
                    };
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        const int k = b.row(j * kPtTile + 32 * q);
                        const uint32_t m = below(see.hi - k) & (~below(see.lo - k) | below(see.few - k));
                        if (__all_sync(0xffffffffu, m == ~0u))
                            continue;
                        float t[32];
                        tmem_ld32(s_cols + 32 * q, t);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            t[c] = (m >> c & 1u) ? t[c] : -INFINITY;
                        tmem_st32(s_cols + 32 * q, t);
                    }
                    tmem_wait_st();
                }
                float s[kPtTile];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    tmem_ld32(s_cols + 32 * q, s + 32 * q);
                tmem_wait_ld();
                float m4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int c = 4; c + 4 < kPtTile; c += 8) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        m4[k] = max3(m4[k], s[c + 2 * k], s[c + 2 * k + 1]);
                }
                const float mxs = max3(max3(m4[0], m4[1], m4[2]), m4[3],
                                       max3(max3(s[kPtTile - 4], s[kPtTile - 3], s[kPtTile - 2]), s[kPtTile - 1], m4[0])) * sc;
                // lazy maximum: O and l are rescaled only when it grows by more than the threshold
                float corr = 1.f;
                if (j == b.jb) {
                    m_run = mxs;
                } else if (mxs > m_run + kPtRescale) {
                    corr = ex2(m_run - mxs);
                    m_run = mxs;
                }
                // (all lanes together: tcgen05 loads and stores under a lane's own condition may never return)
                const bool rescale = __any_sync(0xffffffffu, corr != 1.f);
                const float nm = m_run == -INFINITY ? 0.f : -m_run;   // (no key seen yet)
                const uint64_t sc2 = pk2(sc, sc), nm2 = pk2(nm, nm);
                uint64_t acc[2] = {pk2(0.f, 0.f), pk2(0.f, 0.f)};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float x0, x1;
                        unpk2(fma2(pk2(s[32 * q + 2 * i], s[32 * q + 2 * i + 1]), sc2, nm2), x0, x1);
                        const float p0 = ex2(x0), p1 = ex2(x1);
                        acc[i & 1] = add2(acc[i & 1], pk2(p0, p1));
                        pk[i] = pack_bf16(p0, p1);
                    }
                    tmem_st16(s_cols + 16 * q, pk);
                }
                {
                    float a0, a1, b0, b1;
                    unpk2(acc[0], a0, a1);
                    unpk2(acc[1], b0, b1);
                    l_run = l_run * corr + ((a0 + a1) + (b0 + b1));
                }
                ok = pv_done();
                if (!ok)
                    break;
                if (rescale) {
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        float o[32];
                        tmem_ld32(lane_base + pt_col_o(x) + 32 * q, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] *= corr;
                        tmem_st32(lane_base + pt_col_o(x) + 32 * q, o);
                    }
                }
                tmem_wait_st();
                warp_arrive(kTbP + sb);
            }
            if (!ok)
                break;
            // the row's place, before its output is waited for
            const bool any = b.je > b.jb;   // (else no product was issued, O is not this item's)
            const int row = b.row0 + x * 128 + r, tok = row / G;
            const bool row_ok = x * 128 + r < b.rows;
            const Sees see = sees(a, b.rq, pos);
            const bool some = row_ok && any && see.hi > 0 && (see.few > 0 || see.lo < see.hi);
            const int out_row = row_ok ? (b.l * a.total_q + b.rq.q_off + tok) * a.n_q_heads + b.h * G + (row - tok * G) : -1;
            if (any) {
                if (!mbar_wait_warp(bar(kTbO + x), (uint32_t)o_cnt & 1u, abort_flag)) {
                    ok = false;
                    break;
                }
                ++o_cnt;
                tc_fence_after();
            }
            if (p.splits == 1) {   // the row's output
                if (some && !(l_run > 0.f && l_run < INFINITY))
                    atomicCAS(a.err, kDevOk, kDevBadInput);
                const float inv = 1.f / l_run;
                // half a row at a time, in a loop; two lanes change their rows' 32-byte pieces so that they
                // write 64 bytes in a row
#pragma unroll 1
                for (int hf = 0; hf < 2; ++hf) {
                    uint32_t v[32];
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        float o[32];
                        // (an item without a tile: something, which `some` leaves out)
                        tmem_ld32(lane_base + pt_col_o(x) + 64 * hf + 32 * q, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            v[16 * q + i] = some ? pack_bf16(o[2 * i] * inv, o[2 * i + 1] * inv) : 0u;
                    }
                    // O is read: the next item's first P V is let into it
                    if (any && hf == 1)
                        warp_arrive(kTbOEmpty + x);
                    if (idle)
                        continue;
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (!(i >> 3 & 1)) {
                            const uint32_t got = __shfl_xor_sync(0xffffffffu, (lane & 1) ? v[i] : v[i + 8], 1);
                            v[i] = (lane & 1) ? got : v[i];
                            v[i + 8] = (lane & 1) ? v[i + 8] : got;
                        }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int at = __shfl_sync(0xffffffffu, out_row, (lane & ~1) + i);
                        if (at < 0)
                            continue;
                        uint4 *out = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + (int64_t)at * 128) + 8 * hf +
                                     2 * (lane & 1);
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            uint32_t w[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                w[k] = v[16 * c + 8 * i + k];
                            if (p.out32) {
                                st_global_v8(out + 4 * c, w);
                            } else {
                                out[4 * c] = make_uint4(w[0], w[1], w[2], w[3]);
                                out[4 * c + 1] = make_uint4(w[4], w[5], w[6], w[7]);
                            }
                        }
                    }
                }
                geo_done(item);
            } else {
                const int64_t w = blockIdx.x + (int64_t)item * gridDim.x;
                if (row_ok)
                    part_ml(p.part, w, x)[r] = make_float2(m_run, l_run);
                float4 *po = part_o(p.part, w, x) + r;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (!any)
                        break;
                    float o[32];
                    tmem_ld32(lane_base + pt_col_o(x) + 32 * q, o);
                    tmem_wait_ld();
                    if (row_ok) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            po[(8 * q + i) * 128] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    }
                }
                if (any)
                    warp_arrive(kTbOEmpty + x);
                geo_done(item);
            }
        }
        if (!ok)
            give_up(a.err, abort_flag);
    } else if (warp == 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPtRegsOther));
        pdl_wait_prerequisites();
        bool ok = true;
        int tt = 0, nq[2] = {0, 0};   // loads into the ring, into either query tile
        // item i's geometry into the ring, once the others are done with item i - kPtGeos'
        auto publish = [&](int i) -> bool {
            if (i >= n_items)
                return true;
            const Block b = block_at(a, p, reqs, blockIdx.x + (int64_t)i * gridDim.x);
            const int slot = i % kPtGeos;
            if (i >= kPtGeos && !mbar_wait_warp(bar(kTbGeoFree + slot), (uint32_t)(i / kPtGeos - 1) & 1, abort_flag))
                return false;
            if (lane == 0) {
                *reinterpret_cast<Block *>(smem + kPtOffGeo + slot * kPtGeoBytes) = b;
                mbar_arrive(bar(kTbGeo + slot));
                // its queries, contiguous rows, on their way to L2
                if (b.je > b.jb)
                    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                                     static_cast<const __nv_bfloat16 *>(p.q_rot) +
                                     ((((int64_t)b.lh * a.total_q + b.rq.q_off) * G + b.row0) << 7)),
                                 "r"(b.rows * 256)
                                 : "memory");
            }
            __syncwarp();
            return true;
        };
        const int at_lane = kTwo ? lane : lane >> 1, panel = kTwo ? (int)second : lane & 1;
        ok = second || publish(0);
        for (int item = 0; item < n_items && ok; ++item) {
            if (!(ok = second ? geo_wait(item) : publish(item + 1)))
                break;
            const Block &b = geo(item);
            const int n_loads = 2 * (b.je - b.jb);
            if (n_loads == 0) {
                if (second)
                    geo_done(item);
                continue;
            }
            const int64_t unit = b.unit / 128;
            // tile i of the list: the row of this lane's box and whether it is to be loaded; the same for
            // keys and values
            // (a page's number is asked for a tile ahead of its use)
            const int first = b.first, shift = b.shift, body = b.rq.packed_len;
            int row = 0, at = 0, rows = 0, id = 0, in = 0;
            bool hand = false, load = false, rest = false;
            auto find = [&](int i) {
                auto row_of = [&](int v) -> int { return v < first ? v : v + shift; };
                rest = body > 0 && row_of(i * kPtTile) < body;
                hand = kLoad == kLoadByHand && !rest;
                rows = rest ? kPtTile : p.box;
                at = at_lane * rows;
                const int j0 = row_of(i * kPtTile + at);
                load = !hand && at < kPtTile && (rest || b.some_seen(j0, j0 + rows));
                if (load) {
                    if (rest) {
                        in = b.place(j0);
                    } else {
                        const int pg = page_of(a, j0);
                        in = j0 - pg * a.g.rows;
                        id = page_id(b.rq, ids, pg);
                    }
                }
            };
            find(b.jb);
            for (int i = 0; i <= n_loads; ++i) {
                if (i == 2 && !second) {   // the queries after the first K and V tile
                    if (nq[0] > 0 && !mbar_wait_warp(bar(kTbQEmpty), (uint32_t)(nq[0] - 1) & 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) {
                        const int q0 = (int)(((int64_t)b.lh * a.total_q + b.rq.q_off) * G + b.row0);
                        for (int x = 0; x < b.nx; ++x) {
                            const uint32_t dst = sbase + (uint32_t)(kPtOffQ + x * kPtTileBytes);
                            mbar_expect_tx(bar(kTbQ + x), (uint32_t)kPtTileBytes);
                            tma_load_2d(dst, &tmq, 0, q0 + x * kPtTile, bar(kTbQ + x));
                            tma_load_2d(dst + kPtPanel, &tmq, 64, q0 + x * kPtTile, bar(kTbQ + x));
                        }
                    }
                    ++nq[0];
                    nq[1] += b.nx - 1;
                }
                if (i == n_loads)
                    break;
                const int slot = tt % kPtSlots;
                if (!(i & 1))
                    row = rest ? in : (int)((int64_t)id * (a.g.s_page / 128) + unit + in);
                const uint32_t boxes = (uint32_t)__popc(__ballot_sync(0xffffffffu, load));
                if (tt >= kPtSlots && !mbar_wait_warp(bar(kTbEmpty + slot), (uint32_t)(tt / kPtSlots - 1) & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    if (!hand) {
                        if (!kTwo)
                            mbar_arrive(bar(kTbFull + slot));
                        mbar_expect_tx(bar(kTbFull + slot), boxes * (uint32_t)rows * 128u);
                    } else {
                        mbar_arrive(bar(kTbJob + slot));
                    }
                }
                __syncwarp();   // (the bytes are expected before they land)
                if (load)
                    tma_load_2d(sbase + (uint32_t)(kPtOffKV + slot * kPtTileBytes + panel * kPtPanel + at * 128),
                                (i & 1) ? (rest ? &tmrv : &tmv) : (rest ? &tmrk : &tmk), 64 * panel, row, bar(kTbFull + slot));
                if ((i & 1) && i + 1 < n_loads)
                    find(b.jb + (i >> 1) + 1);
                ++tt;
            }
            if (ok && second)
                geo_done(item);
        }
        if (!ok)
            give_up(a.err, abort_flag);
        // copies in flight land before the CTA leaves
        if (lane == 0) {
            for (int k = tt > kPtSlots ? tt - kPtSlots : 0; k < tt; ++k)
                mbar_drain(bar(kTbFull + k % kPtSlots), (uint32_t)(k / kPtSlots) & 1);
            for (int x = 0; x < 2; ++x)
                if (nq[x] > 0)
                    mbar_drain(bar(kTbQ + x), (uint32_t)(nq[x] - 1) & 1);
        }
        __syncwarp();
    } else if (warp == 9) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPtRegsOther));
        pdl_wait_prerequisites();
        const uint32_t lead = elect_one();
        int tt = 0;
        // bit x: the parity of the next phase of P (O, Q) barrier x; O x holds an output
        uint32_t p_par = 0, o_par = 0, q_par = 0, o_used = 0;
        bool ok = true;
        const uint64_t d_k = sdesc(sbase, 16, 1024), d_v = sdesc(sbase, kPtPanel, 1024);
        const uint32_t lo_k = (uint32_t)d_k, hi_k = (uint32_t)(d_k >> 32), lo_v = (uint32_t)d_v, hi_v = (uint32_t)(d_v >> 32);
        auto wait_kv = [&](int k) -> bool {
            if (!mbar_wait_warp(bar(kTbFull + k % kPtSlots), (uint32_t)(k / kPtSlots) & 1, abort_flag))
                return false;
            tc_fence_after();
            return true;
        };
        // S = Q_x K^T, with K the ring's load k, into buffer sb
        auto issue_s = [&](int x, int k, int sb) {
            const uint32_t qa = lo_k + ((uint32_t)(kPtOffQ + x * kPtTileBytes) >> 4);
            const uint32_t kb = lo_k + ((uint32_t)(kPtOffKV + (k % kPtSlots) * kPtTileBytes) >> 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t off = (uint32_t)((i >> 2) * kPtPanel + (i & 3) * 32) >> 4;
                mma_ss(lead, tmem + pt_col_s(sb), desc_with_lo(qa + off, hi_k), desc_with_lo(kb + off, hi_k), kPtIdescS, i > 0);
            }
            umma_commit(lead, bar(kTbS + sb));
        };
        auto issue_pv = [&](int x, int k, uint32_t acc0, int sb) {
            const uint32_t vb = lo_v + ((uint32_t)(kPtOffKV + (k % kPtSlots) * kPtTileBytes) >> 4);
#pragma unroll
            for (int i = 0; i < kPtTile / 16; ++i)
                mma_ts(lead, tmem + pt_col_o(x), tmem + pt_col_s(sb) + 8 * i, desc_with_lo(vb + ((i * 2048) >> 4), hi_v), kPtIdescPV,
                       i > 0 ? 1u : acc0);
        };
        for (int item = 0; item < n_items && ok; ++item) {
            if (!geo_wait(item)) {
                ok = false;
                break;
            }
            const Block &b = geo(item);
            const int K = b.je - b.jb;
            if (K == 0) {
                geo_done(item);
                continue;
            }
            // V tile i of the item has rows that no query sees, which have to be zeroed: only one where the
            // first rows or the window begin or end
            const int j_cut = b.first / kPtTile, j_end = (b.any.hi - b.shift) / kPtTile;
            auto holes = [&](int i) -> bool {
                const int j = b.jb + i, v0 = j * kPtTile, v1 = v0 + kPtTile;
                if (j > j_cut && j < j_end)
                    return false;
                const bool all = b.cut(j) ? b.all_seen(v0, b.first) && b.all_seen(b.first + b.shift, v1 + b.shift)
                                          : b.all_seen(b.row(v0), b.row(v0) + kPtTile);
                return !all && !by_hand<kLoad>(b, j) && !b.restored(j);
            };
            // V tile i: landed, such rows zeroed
            auto wait_v = [&](int i, bool zero) -> bool {
                if (!wait_kv(tt + 2 * i + 1))
                    return false;
                if (zero) {
                    const int v0 = (b.jb + i) * kPtTile;
                    const uint32_t v = sbase + (uint32_t)(kPtOffKV + ((tt + 2 * i + 1) % kPtSlots) * kPtTileBytes);
                    for (int c = lane; c < kPtTile * 8; c += 32)
                        if (!b.any(b.row(v0 + (c >> 3)))) {
                            st_shared_v4(v + 16u * (uint32_t)c, 0u, 0u, 0u, 0u);
                            st_shared_v4(v + kPtPanel + 16u * (uint32_t)c, 0u, 0u, 0u, 0u);
                        }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                return true;
            };
            auto o_free = [&](int x) -> bool {
                if (o_used >> x & 1u) {
                    if (!mbar_wait_warp(bar(kTbOEmpty + x), o_par >> x & 1u, abort_flag))
                        return false;
                    o_par ^= 1u << x;
                    o_used ^= 1u << x;
                }
                return true;
            };
            if (!mbar_wait_warp(bar(kTbQ), q_par & 1u, abort_flag)) {
                ok = false;
                break;
            }
            q_par ^= 1u;
            tc_fence_after();
            if constexpr (kOne) {
                auto s_of = [&](int i) -> bool {   // S of key tile i into buffer i & 1
                    if (!wait_kv(tt + 2 * i))
                        return false;
                    issue_s(0, tt + 2 * i, i & 1);
                    umma_commit(lead, bar(kTbEmpty + (tt + 2 * i) % kPtSlots));
                    if (i + 1 == K)
                        umma_commit(lead, bar(kTbQEmpty));
                    return true;
                };
                ok = s_of(0) && (K == 1 || s_of(1)) && o_free(0);
                for (int i = 0; i < K && ok; ++i) {
                    const int sb = i & 1;
                    const bool zero = holes(i);
                    if (!mbar_wait_warp(bar(kTbP + sb), (p_par >> sb) & 1u, abort_flag) || !wait_v(i, zero)) {
                        ok = false;
                        break;
                    }
                    p_par ^= 1u << sb;
                    tc_fence_after();
                    issue_pv(0, tt + 2 * i + 1, i > 0, sb);
                    umma_commit(lead, bar(i + 1 < K ? kTbPv : kTbO));
                    umma_commit(lead, bar(kTbEmpty + (tt + 2 * i + 1) % kPtSlots));
                    ok = i + 2 >= K || s_of(i + 2);
                }
                o_used = 1u;
            } else {
            ok = wait_kv(tt);
            if (!ok)
                break;
            // (into S at once: O, which the epilogue before may still read, is the first P V's affair)
#pragma unroll
            for (int x = 0; x < 2; ++x)
                if (x < b.nx) {
                    if (x == 1) {   // (its queries land behind tile A's)
                        if (!(ok = mbar_wait_warp(bar(kTbQ + 1), q_par >> 1, abort_flag)))
                            break;
                        q_par ^= 2u;
                        tc_fence_after();
                    }
                    issue_s(x, tt, x);
                }
            if (!ok)
                break;
            umma_commit(lead, bar(kTbEmpty + tt % kPtSlots));
            if (K == 1)
                umma_commit(lead, bar(kTbQEmpty));
            const bool two = b.nx == 2;
            for (int i = 0; i < K && ok; ++i) {
                const bool more = i + 1 < K, zero = holes(i);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (x == 1 && !two)
                        break;
                    // (the probabilities last: nothing stands between them and the product)
                    if ((x == 0 && !wait_v(i, zero)) || (i == 0 && !o_free(x)) ||
                        !mbar_wait_warp(bar(kTbP + x), (p_par >> x) & 1u, abort_flag)) {
                        ok = false;
                        break;
                    }
                    p_par ^= 1u << x;
                    tc_fence_after();
                    issue_pv(x, tt + 2 * i + 1, i > 0, x);
                    if (!more) {
                        umma_commit(lead, bar(kTbO + x));
                        o_used |= 1u << x;
                    } else {
                        if (x == 0 && !wait_kv(tt + 2 * i + 2)) {
                            ok = false;
                            break;
                        }
                        issue_s(x, tt + 2 * i + 2, x);
                    }
                }
                if (!ok)
                    break;
                if (i + 2 == K)
                    umma_commit(lead, bar(kTbQEmpty));   // the item's last S is issued
                umma_commit(lead, bar(kTbEmpty + (tt + 2 * i + 1) % kPtSlots));
                if (more)
                    umma_commit(lead, bar(kTbEmpty + (tt + 2 * i + 2) % kPtSlots));
            }
            }
            tt += 2 * K;
            geo_done(item);
        }
        if (!ok)
            give_up(a.err, abort_flag);
        umma_commit(lead, bar(kTbDrain));
        mbar_drain(bar(kTbDrain), 0);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPtRegsOther));
        pdl_wait_prerequisites();
        bool ok = true;
        int tt = 0;
        uint32_t jobs = 0;   // bit s: the parity of slot s's next job
        // Up to three tiles' copies are in flight: their slots, the oldest in the lowest byte.  One is passed
        // on when a fourth is asked for, or as soon as there is nothing to do: the products may wait for it.
        uint32_t flight = 0;
        int n_flight = 0;
        auto landed = [&](int keep) {
            if (keep == 0)
                copies_wait<0>();
            else
                copies_wait<2>();
            fence_proxy_async_smem();
            __syncwarp();
            for (; n_flight > keep; --n_flight, flight >>= 8)
                if (lane == 0)
                    mbar_arrive(bar(kTbFull + (int)(flight & 255u)));
        };
        int64_t at[2] = {-1, -1};   // of this lane's rows of the tile: elements from the unit's start; < 0: zeros
        for (int item = 0; item < n_items && ok; ++item) {
            if (!geo_wait(item)) {
                ok = false;
                break;
            }
            const Block &b = geo(item);
            const int n_loads = 2 * (b.je - b.jb);
            for (int i = 0; i < n_loads; ++i, ++tt) {
                const int slot = tt % kPtSlots, t = b.jb + (i >> 1);
                if (!by_hand<kLoad>(b, t))
                    continue;
                if (n_flight > 0 && !mbar_test_warp(bar(kTbJob + slot), (jobs >> slot) & 1u))
                    landed(0);
                if (!mbar_wait_warp(bar(kTbJob + slot), (jobs >> slot) & 1u, abort_flag)) {
                    ok = false;
                    break;
                }
                jobs ^= 1u << slot;
                if (!(i & 1)) {   // (a row's place once, for its key and its value)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int j = b.row(t * kPtTile + 64 * (warp - 10) + 32 * k + lane);
                        at[k] = -1;
                        if (b.any(j)) {
                            const int pg = page_of(a, j);
                            at[k] = (int64_t)page_id(b.rq, ids, pg) * a.g.s_page + (int64_t)(j - pg * a.g.rows) * 128;
                        }
                    }
                }
                const uint32_t tile = sbase + (uint32_t)(kPtOffKV + slot * kPtTileBytes);
                const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>((i & 1) ? a.g.v : a.g.k);
                const int ch = lane & 15;
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll 4
                    for (int y = 0; y < 16; ++y) {
                        const int row = 64 * (warp - 10) + 32 * k + 2 * y + (lane >> 4);
                        const int64_t o = __shfl_sync(0xffffffffu, at[k], 2 * y + (lane >> 4));
                        copy16(tile + (uint32_t)((ch >> 3) * kPtPanel + row * 128 + (((ch & 7) ^ (row & 7)) << 4)),
                               src + (o >= 0 ? b.unit + o + 8 * ch : 0), o >= 0);
                    }
                copies_end();
                flight |= (uint32_t)slot << 8 * n_flight;
                if (++n_flight == 3)
                    landed(2);
            }
            if (ok)
                landed(0);
            geo_done(item);
        }
        copies_wait<0>();
        if (!ok)
            give_up(a.err, abort_flag);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, kPtTmemCols);
    }
}

// Packed rows of the slice's units as bf16 rows, for the requests of more than
// kPageFewRows query rows.  One CTA: the keys or the values of one tile of 128 rows, a
// warp a block of 32.  Rows behind packed_len in the last tile are copied from the pages,
// rows that no query sees are zeros.  Bound by HBM: 0.75 GB read and written in 121 us.
__global__ void __launch_bounds__(128)
    k_page_restore(const __grid_constant__ PageArgs a, const __grid_constant__ PageTcArgs p, const __grid_constant__ PageTable pt)
{
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const DevPageReq *reqs = a.reqs ? a.reqs : pt.reqs;
    const int32_t *ids = a.reqs ? a.ids : pt.ids;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = lane >> 2, c = lane & 3;
    const int part = (int)(blockIdx.x & 1u), tile = (int)((blockIdx.x >> 1) % (unsigned)p.unit_tiles);
    const int lh_s = (int)((blockIdx.x >> 1) / (unsigned)p.unit_tiles), lh = p.lh_base + lh_s;
    int lo = 0, hi = a.n_reqs - 1;
    while (lo < hi) {   // the last request whose first tile is <= it (one with tiles)
        const int mid = (lo + hi + 1) >> 1;
        if (reqs[mid].tile0 <= tile)
            lo = mid;
        else
            hi = mid - 1;
    }
    const DevPageReq rq = reqs[lo];
    const Sees any = sees_any(a, rq);
    const int j0 = rest_tiles(any.hi, any.lo, any.few, rq.packed_len).tile(tile - rq.tile0) * kPtTile + 32 * warp;
    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(part ? p.rest_v : p.rest_k) +
                                           ((int64_t)(lh_s * p.unit_tiles + tile) * kPtTile + 32 * warp) * 128);
    if (j0 < rq.packed_len && (j0 < any.few || (j0 < any.hi && j0 + 32 > any.lo))) {
        const uint8_t *src = a.g.packed + packed_block(a, rq, ids, lh, j0);
        const int place = part ? 4 * (lane & 7) + (lane >> 3) : lane;
        uint4 codes[4];
        uint2 sc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            codes[i] = __ldg(reinterpret_cast<const uint4 *>(src + codes_at(i, part) + 16 * place));
            sc[i] = __ldg(reinterpret_cast<const uint2 *>(src + scales_at(8 * i + n, part)));
            if (!any(j0 + 8 * i + n))   // (its scales may be NaN)
                sc[i] = make_uint2(0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w[4] = {codes[i].x, codes[i].y, codes[i].z, codes[i].w};
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const uint32_t s = prmt(g < 2 ? sc[i].x : sc[i].y, 0u, (g & 1) ? 0x3232u : 0x1010u);
                dst[(8 * i + n) * 16 + 4 * g + c] = restore8(w[g], part, s, lane);
            }
        }
        return;
    }
    const int l = lh / a.n_kv_heads, h = lh - l * a.n_kv_heads;
    const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(part ? a.g.v : a.g.k) + l * a.g.s_layer + h * a.g.s_head;
    const int ch = lane & 15;
#pragma unroll 4
    for (int y = 0; y < 16; ++y) {
        const int row = 2 * y + (lane >> 4), j = j0 + row;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (any(j) && j >= rq.packed_len) {
            const int pg = page_of(a, j);
            v = __ldg(reinterpret_cast<const uint4 *>(src + (int64_t)page_id(rq, ids, pg) * a.g.s_page + (int64_t)(j - pg * a.g.rows) * 128) + ch);
        }
        dst[row * 16 + ch] = v;
    }
}

// The partial results of a block's stretches, one after the other.  A CTA: 16 columns of a
// 128-row tile, a thread a row, whose loads are all in flight at once.  (128 columns a
// CTA: 274 us a call for 64 tokens x 4 heads on 33,000 rows, 64 units; 16 columns: 243.)
__global__ void __launch_bounds__(128)
    k_page_join(const __grid_constant__ PageArgs a, const __grid_constant__ PageTcArgs p, const __grid_constant__ PageTable pt)
{
    pdl_wait_prerequisites();
    const DevPageReq *reqs = a.reqs ? a.reqs : pt.reqs;
    const int G = a.n_q_heads / a.n_kv_heads, part = (int)(blockIdx.x & 7u), x = (int)(blockIdx.x >> 3 & 1u), r = threadIdx.x;
    const int64_t w0 = (int64_t)(blockIdx.x >> 4) * p.splits;
    const Block b = block_at(a, p, reqs, w0);
    if (x * 128 + r >= b.rows)
        return;
    const int tok = (b.row0 + x * 128 + r) / G, g = b.row0 + x * 128 + r - tok * G;
    const Sees see = sees(a, b.rq, b.rq.pos0 + tok);
    const bool some = see.hi > 0 && (see.few > 0 || see.lo < see.hi);
    float m = -INFINITY, L = 0.f;
    for (int i = 0; i < p.splits; ++i)
        m = fmaxf(m, part_ml(p.part, w0 + i, x)[r].x);
    float4 v[4] = {};
#pragma unroll 2
    for (int i = 0; i < p.splits; ++i) {
        const float2 ml = part_ml(p.part, w0 + i, x)[r];
        if (ml.x == -INFINITY && ml.y == 0.f)   // (nothing seen: its O may not be written)
            continue;
        const float f = ml.x == -INFINITY ? 1.f : ex2(ml.x - m);   // (a stretch of NaN scores: a sum of NaN under -inf)
        L = fmaf(ml.y, f, L);
        const float4 *o = part_o(p.part, w0 + i, x) + 4 * part * 128 + r;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float4 y = o[c * 128];
            v[c].x = fmaf(y.x, f, v[c].x);
            v[c].y = fmaf(y.y, f, v[c].y);
            v[c].z = fmaf(y.z, f, v[c].z);
            v[c].w = fmaf(y.w, f, v[c].w);
        }
    }
    if (some && part == 0 && !(L > 0.f && L < INFINITY))
        atomicCAS(a.err, kDevOk, kDevBadInput);
    const float inv = some ? 1.f / L : 0.f;
    const int l = b.lh / a.n_kv_heads, h = b.lh - l * a.n_kv_heads;
    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) +
                                           (((int64_t)l * a.total_q + b.rq.q_off + tok) * a.n_q_heads + h * G + g) * 128) + 2 * part;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const float4 y = v[2 * c], z = v[2 * c + 1];
        dst[c] = some ? make_uint4(pack_bf16(y.x * inv, y.y * inv), pack_bf16(y.z * inv, y.w * inv), pack_bf16(z.x * inv, z.y * inv),
                                   pack_bf16(z.z * inv, z.w * inv))
                      : make_uint4(0u, 0u, 0u, 0u);
    }
}

// The query heads of the requests of more than kPageFewRows rows, turned and packed:
// [L][H_kv][T][G][D].  8 threads a (layer, token, kv-head), in the queries' order.
__global__ void __launch_bounds__(128)
    k_page_queries(const __grid_constant__ PageArgs a, const __grid_constant__ PageTable pt, __nv_bfloat16 *__restrict__ q_rot)
{
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const DevPageReq *reqs = a.reqs ? a.reqs : pt.reqs;
    const int G = a.n_q_heads / a.n_kv_heads, H = a.n_kv_heads, j = threadIdx.x & 7;
    const int64_t item = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 3);
    if (item >= (int64_t)a.n_layers * a.total_q * H)
        return;
    const int64_t lt = item / H;
    const int h = (int)(item - lt * H), l = (int)(lt / a.total_q), tok = (int)(lt - (int64_t)l * a.total_q);
    int lo = 0, hi = a.n_reqs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (reqs[mid].q_off <= tok)
            lo = mid;
        else
            hi = mid - 1;
    }
    const DevPageReq &rq = reqs[lo];
    if (rq.q_len * G <= kPageFewRows)
        return;
    const bool il = a.interleaved != 0;
    float cs[8], sn[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float2 v = rope_cs(a.rope, 64, rq.pos0 + tok - rq.q_off, rope_pair(il, 128, 8, j, e));
        cs[e] = v.x;
        sn[e] = v.y;
    }
    const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(a.q) + item * G * 128 + 8 * j;
    __nv_bfloat16 *dst = q_rot + (((int64_t)l * H + h) * a.total_q + tok) * G * 128 + 8 * j;
#pragma unroll 4
    for (int g = 0; g < G; ++g) {
        uint4 x = __ldg(reinterpret_cast<const uint4 *>(src + g * 128)), y = __ldg(reinterpret_cast<const uint4 *>(src + g * 128 + 64));
        if (il)
            rotate_bf16x8_il(x, y, cs, sn);
        else
            rotate_bf16x8(x, y, cs, sn);
        *reinterpret_cast<uint4 *>(dst + g * 128) = x;
        *reinterpret_cast<uint4 *>(dst + g * 128 + 64) = y;
    }
}

cudaError_t launch_page_queries(const PageArgs &a, const PageTable &t, void *q_rot, cudaStream_t s)
{
    const int64_t triples = (int64_t)a.n_layers * a.total_q * a.n_kv_heads;
    return launch_pdl(k_page_queries, (triples + 15) / 16, 128, 0, true, s, a, t, static_cast<__nv_bfloat16 *>(q_rot));
}

cudaError_t launch_page_tc(const PageArgs &a, const PageTcArgs &p, const PageTable &t, const PageTcMaps &m, int lh_count, int n_sms,
                           cudaStream_t s)
{
    static std::atomic<bool> attr_set[64] = {};   // per device (host threads may race: same value)
    decltype(&k_page_attention<false, 0>) const kernels[5] = {
        k_page_attention<false, kLoadOne>, k_page_attention<false, kLoadTwo>, k_page_attention<false, kLoadByHand>,
        k_page_attention<true, kLoadTwo>, k_page_attention<true, kLoadByHand>};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev >= 64 || !attr_set[dev].load(std::memory_order_acquire)) {
        for (auto *k : kernels) {
            cudaFuncAttributes fa{};
            if ((e = cudaFuncGetAttributes(&fa, k)) != cudaSuccess)
                return e;
            // the roles' register counts draw on what the launch holds: exactly this many
            if (fa.numRegs != kPtRegsLaunch)
                return cudaErrorInvalidConfiguration;
            if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kPtSmem)) != cudaSuccess)
                return e;
        }
        if (dev < 64)
            attr_set[dev].store(true, std::memory_order_release);
    }
    auto map = [](const void *x) -> const CUtensorMap & { return *static_cast<const CUtensorMap *>(x); };
    if (p.unit_tiles > 0)
        e = launch_pdl(k_page_restore, 2 * (int64_t)lh_count * p.unit_tiles, 128, 0, true, s, a, p, t);
    const int load = p.box == 0 ? kLoadByHand : p.one_tile || p.box <= 32 ? kLoadTwo : kLoadOne;
    if (e == cudaSuccess)
        e = launch_pdl(kernels[load + (p.one_tile ? 2 : 0)], std::min<int64_t>(n_sms, p.total), kPtThreads, kPtSmem, true, s, map(m.q),
                       map(m.k), map(m.v), map(m.rest_k), map(m.rest_v), a, p, t);
    if (e == cudaSuccess && p.splits > 1)
        e = launch_pdl(k_page_join, 16 * (p.total / p.splits), 128, 0, true, s, a, p, t);
    return e;
}

}  // namespace kvr
