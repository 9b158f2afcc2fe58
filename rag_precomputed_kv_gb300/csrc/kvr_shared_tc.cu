// kvr_shared_tc.cu -- query attention over a prefix shared by a group of
// requests, on the tensor cores (bf16, head_dim 128).
//
// O_r = (sum_j e^{s_rj} v_j) / (sum_j e^{s_rj}) over the shared prefix rows and
// the request's own rows (CoinRAG blog section 2.3: KV_M(q; C_ctx), with C_ctx
// the same for the whole group).  The sums over a set of keys, each with its
// own maximum m (sum e^{s - m} v, sum e^{s - m}), add after scaling by
// e^{m - max}, so the two parts are computed apart:
//
//   k_shared_prologue  rotates the query heads at P_g + S_b + t into a packed
//                      scratch [layer][kv-head][token][G][D], and appends the
//                      keys (rotated) and values at own row S_b + t.
//   k_shared_prefix    the prefix part.  The packed rows of a whole group are
//                      consecutive: M = tokens of the group x G rows meet each
//                      prefix tile once, in blocks of up to 256 rows.
//                      tcgen05, as the query-prefill attention: 128-row tiles
//                      A and B per CTA, S and P and O in TMEM.  The work, all
//                      (block, key tile) pairs of the call in a row, is cut in
//                      equal stretches, one per SM; a block that a stretch ends
//                      in has several partial results.
//   k_shared_whole     the same for whole blocks, whose rows' own keys follow
//                      the prefix's, tile by tile, request by request; it
//                      writes the output.  Nothing else is launched then.
//   k_shared_own_*     the own part, and the sum of everything: the own rows
//                      through register-resident warp MMAs (as the decode
//                      step), then the prefix's partial results are added and
//                      the output written.
//
// A block of at most 128 rows (a decode step of a few requests) uses tile A
// alone: its time is the reads of K and V.  (Both tiles on the same rows and
// alternate key tiles, so that one's softmax overlaps the other's: 736 us
// against 695 for 64 rows on 33,248 prefix rows and 256 units, 105 against 95
// for 7 rows on 8,256 and 112 units: twice the partial results, for nothing.)
//
// Values behind the last row are zeroed in shared memory before the P V product
// that reaches them (a masked key's weight is 0, but 0 x NaN is NaN), so the
// blocks' spare rows are neither read as data nor written; an own tile's
// product leaves the O rows of other requests out.
//
// Measured on whole calls (bf16, head_dim 128): 64 rows on 33,248 prefix rows,
// 256 units: k_shared_prefix 606 us, 7.2 TB/s of K and V; 256 rows on 8,256, 288
// units: 213 us, 1.46 PFLOP/s, and 166 us for 64 requests' own rows (4.6 TB/s);
// 6,328 rows on 2,592, 112 units: k_shared_whole 850 us, 1.12 PFLOP/s, behind 80
// us of k_shared_prologue (5.8 TB/s).
//
// Rounded to bf16 on the way, as the query prefill and the decode step do it: the
// rotated queries (the cached keys are) and each probability, because both are
// operands of a product with bf16 keys or values.  With the output's own rounding
// that is 0.0029 of the output's norm, against 0.0017 for the last alone; two
// bf16 terms for the queries would add half of all products, for the
// probabilities another half.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>
#include <utility>

#include "kvr_decode_common.cuh"
#include "kvr_tc_common.cuh"

namespace kvr {

namespace {

using namespace tc;

constexpr int kSpThreads = 384;
constexpr int kSpRegsLaunch = 168, kSpRegsSoftmax = 200, kSpRegsOther = 104;
static_assert(2 * 128 * kSpRegsSoftmax + 128 * kSpRegsOther <= kSpThreads * kSpRegsLaunch, "register split");
constexpr int kSpD = 128;
constexpr int kSpTile = 128;                        // keys per tile, rows per query tile
constexpr int kSpSlots = 5;                         // K/V ring
constexpr int kSpTileBytes = kSpTile * kSpD * 2;    // 32 KB
constexpr int kSpPanel = kSpTileBytes / 2;
constexpr int kSpTmemCols = 512;
__host__ __device__ constexpr uint32_t sp_col_s(int x) { return 128u * (uint32_t)x; }
__host__ __device__ constexpr uint32_t sp_col_o(int x) { return 256u + 128u * (uint32_t)x; }
constexpr float kSpRescale = 8.0f;

constexpr int kSpOffQ = 0;
constexpr int kSpOffKV = 2 * kSpTileBytes;
constexpr int kSpOffBar = kSpOffKV + kSpSlots * kSpTileBytes;
constexpr int kSbFull = 0, kSbEmpty = kSbFull + kSpSlots, kSbS = kSbEmpty + kSpSlots, kSbP = kSbS + 2, kSbO = kSbP + 2,
              kSbOEmpty = kSbO + 2, kSbQ = kSbOEmpty + 2, kSbQEmpty = kSbQ + 1, kSbDrain = kSbQEmpty + 1,
              kSbNum = kSbDrain + 1;
constexpr int kSpOffMisc = kSpOffBar + 8 * kSbNum;
constexpr int kSpSmem = kSpOffMisc + 16 + 1024;     // + alignment slack
static_assert(kSpSmem <= 227 * 1024, "shared memory budget");

constexpr uint32_t kSpIdescS = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kSpTile >> 3) << 17) |
                               ((uint32_t)(kSpTile >> 4) << 24);
constexpr uint32_t kSpIdescPV = kSpIdescS | (1u << 16);   // V is MN-major

// A partial result of one block and one CTA: per tile x, O as float4
// [column / 4][row] (lanes are rows: coalesced), then (max, sum) [row].
constexpr int64_t kPartO = 2 * 128 * 128;                        // floats
constexpr int64_t kPartFloats = kPartO + 2 * 128 * 2;
static_assert(kPartFloats * 4 == kSharedPartBytes, "partial result layout");

__device__ __forceinline__ float4 *part_o(float *part, int64_t slot, int x)
{
    return reinterpret_cast<float4 *>(part + slot * kPartFloats) + x * (128 * 32);
}
__device__ __forceinline__ float2 *part_ml(float *part, int64_t slot, int x)
{
    return reinterpret_cast<float2 *>(part + slot * kPartFloats + kPartO) + x * 128;
}

// Stretch c of the call's `total` (block, key tile) pairs starts here.
__device__ __forceinline__ int64_t stretch_start(int64_t total, int n, int c) { return total * c / n; }
// The stretch that holds pair w: the last c with total * c / n <= w, that is
// total * c < n (w + 1); `ratio` = n / total gives it within one.
__device__ __forceinline__ int stretch_of(int64_t total, int n, float ratio, int64_t w)
{
    int c = min((int)((float)w * ratio), n - 1);
    const int64_t lim = (int64_t)n * (w + 1);
    while (total * c >= lim)
        --c;
    while (total * (c + 1) < lim)
        ++c;
    return c;
}

// One block's part in a CTA's stretch.
struct Seg {
    DevGroup g;
    int lh;          // (layer, kv-head), within the call's slice
    int row0;        // first packed row of the block in the group
    int rows;        // rows of the block (<= 256)
    int nx;          // its 128-row tiles: A, or A and B
    int jb, je;      // key tiles
    int64_t item;    // block index in the call
    int64_t next;    // the stretch's next pair (whole: the CTA's next block)

    __device__ __forceinline__ void set_rows(int blk)
    {
        row0 = blk * 256;
        rows = min(256, g.rows - row0);
        nx = rows > 128 ? 2 : 1;
    }
};

__device__ __forceinline__ Seg seg_at(const SharedPrefixArgs &a, const DevGroup *groups, int64_t w, int64_t w_end)
{
    Seg s;
    s.lh = (int)(w / a.unit_pairs);
    const int64_t in_unit = w - (int64_t)s.lh * a.unit_pairs;
    int lo = 0, hi = a.n_groups - 1;
    while (lo < hi) {   // the last group whose first pair in the unit is <= w (one with tiles)
        const int mid = (lo + hi + 1) >> 1;
        if (groups[mid].w0 <= in_unit)
            lo = mid;
        else
            hi = mid - 1;
    }
    s.g = groups[lo];
    const int blk = (int)((in_unit - s.g.w0) / s.g.nt);
    s.jb = (int)(in_unit - s.g.w0 - (int64_t)blk * s.g.nt);
    s.je = (int)min((int64_t)s.g.nt, s.jb + (w_end - w));
    s.next = w + (s.je - s.jb);
    s.item = (int64_t)s.lh * a.unit_blocks + s.g.item0 + blk;
    s.set_rows(blk);
    return s;
}

// The whole blocks of CTA c of n: runs of a.run blocks go round the CTAs, what is
// left over is cut in equal stretches.
__device__ __forceinline__ int64_t blocks_of(const SharedPrefixArgs &a, int n, int c)
{
    const int64_t rounds = a.total / ((int64_t)n * a.run), rest = a.total - rounds * n * a.run;
    return rounds * a.run + stretch_start(rest, n, c + 1) - stretch_start(rest, n, c);
}
// The w-th of them, with all tiles of the prefix.
__device__ __forceinline__ Seg block_at(const SharedPrefixArgs &a, const DevGroup *groups, int64_t w, int n, int c)
{
    Seg s;
    const int64_t rounds = a.total / ((int64_t)n * a.run), q = w / a.run;
    const int64_t i = q < rounds ? (q * n + c) * a.run + (w - q * a.run)
                                 : rounds * n * a.run + stretch_start(a.total - rounds * n * a.run, n, c) + (w - rounds * a.run);
    s.lh = (int)(i / a.unit_blocks);
    const int64_t in_unit = i - (int64_t)s.lh * a.unit_blocks;
    int lo = 0, hi = a.n_groups - 1;
    while (lo < hi) {   // the last group whose first block in the unit is <= i (one with blocks)
        const int mid = (lo + hi + 1) >> 1;
        if (groups[mid].item0 <= in_unit)
            lo = mid;
        else
            hi = mid - 1;
    }
    s.g = groups[lo];
    s.jb = 0;
    s.je = s.g.nt;
    s.next = w + 1;
    s.item = i;
    s.set_rows((int)(in_unit - s.g.item0));
    return s;
}

// The own key tiles that a whole block meets: request by request, those of the
// requests that its rows belong to, as far as the block's last row sees.
struct OwnTiles {
    int b, k;        // request, key tile
    int t_end;       // token behind the block's last

    __device__ __forceinline__ int keys(const DevShared &r) const { return r.own + min(r.q_len, t_end - r.q_off); }
    __device__ __forceinline__ void skip_empty(const DevShared *reqs, int n_reqs)
    {
        while (b < n_reqs && reqs[b].q_len == 0)
            ++b;
    }
    // the block's first tile; returns how many there are
    __device__ __forceinline__ int first(const DevShared *reqs, int n_reqs, const Seg &s, int G)
    {
        const int t0 = s.g.q_off + s.row0 / G;
        t_end = s.g.q_off + (s.row0 + s.rows - 1) / G + 1;
        int lo = 0, hi = n_reqs - 1;
        while (lo < hi) {   // the last request that starts at or before the first token
            const int mid = (lo + hi + 1) >> 1;
            if (reqs[mid].q_off <= t0)
                lo = mid;
            else
                hi = mid - 1;
        }
        int n = 0;
        for (b = lo; b < n_reqs && reqs[b].q_off < t_end; ++b)
            n += reqs[b].q_len > 0 ? (keys(reqs[b]) + kSpTile - 1) / kSpTile : 0;
        b = lo;
        k = 0;
        return n;
    }
    __device__ __forceinline__ void next(const DevShared *reqs, int n_reqs)
    {
        if (++k * kSpTile >= keys(reqs[b])) {
            ++b;
            k = 0;
            skip_empty(reqs, n_reqs);
        }
    }
};

// kWhole: whole blocks, whose own keys follow the prefix's, and whose rows are
// written as the output, else stretches of pairs and partial results of the
// prefix.  Whole blocks go round the CTAs in short runs: those of a unit, which
// read the same prefix, run at the same time (all of a CTA's blocks in a row: 1.7
// GB read from DRAM for 0.25 GB of prefix and queries).
template <bool kWhole>
__device__ __forceinline__ void prefix_part(const CUtensorMap &tmq, const CUtensorMap &tmk, const CUtensorMap &tmv,
                                            const SharedPrefixArgs &a, const DevGroup *groups, const CUtensorMap &tmok,
                                            const CUtensorMap &tmov, const SharedArgs *sa, const DevShared *reqs)
{
    extern __shared__ uint8_t sp_smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(sp_smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    auto bar = [&](int i) { return sbase + kSpOffBar + 8u * (uint32_t)i; };
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kSpOffMisc + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t w_begin = kWhole ? 0 : stretch_start(a.total, (int)gridDim.x, (int)blockIdx.x);
    const int64_t w_end = kWhole ? blocks_of(a, (int)gridDim.x, (int)blockIdx.x)
                                 : stretch_start(a.total, (int)gridDim.x, (int)blockIdx.x + 1);
    auto seg = [&](int64_t w, OwnTiles &ot) -> Seg {
        if constexpr (kWhole) {
            Seg s = block_at(a, groups, w, (int)gridDim.x, (int)blockIdx.x);
            s.je += ot.first(reqs, sa->n_reqs, s, a.group);
            return s;
        } else {
            return seg_at(a, groups, w, w_end);
        }
    };

    if (threadIdx.x == 0) {
        for (int i = 0; i < kSbNum; ++i)
            mbar_init(bar(i), (i >= kSbP && i < kSbP + 2) || (i >= kSbOEmpty && i < kSbOEmpty + 2) ? 128u : 1u);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 9)
        tmem_alloc(sbase + kSpOffMisc, kSpTmemCols);
    if (warp == 8 && lane == 0) {
        prefetch_tmap(&tmq);
        prefetch_tmap(&tmk);
        prefetch_tmap(&tmv);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + kSpOffMisc);

    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSpRegsSoftmax));
        pdl_wait_prerequisites();   // (the partial results' scratch may still be read by the call before)
        // the own part may be set up now, and load what the prologue, now done, wrote
        if (!kWhole && blockIdx.x == 0 && threadIdx.x == 0)
            relay_store(a.relay + 1, a.call);
        pdl_launch_dependents();
        const int x = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const float sc = a.scale_log2;
        int s_cnt = 0, o_cnt = 0;
        bool ok = true;
        for (int64_t w = w_begin; w < w_end && ok;) {
            OwnTiles ot;
            const Seg sg = seg(w, ot);
            w = sg.next;
            if (x >= sg.nx)
                continue;
            const bool row_ok = x * 128 + r < sg.rows;
            // a warp without rows of its own only keeps the barriers going: what it
            // leaves in its lanes of P meets its own lanes of O alone
            const bool idle = x * 128 + (warp & 3) * 32 >= sg.rows;
            const int tok = kWhole ? sg.g.q_off + (sg.row0 + x * 128 + r) / a.group : 0;
            float m_run = -INFINITY, l_run = 0.f;
            for (int j = sg.jb; j < sg.je; ++j) {
                if (!mbar_wait_warp(bar(kSbS + x), (uint32_t)s_cnt & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                ++s_cnt;
                tc_fence_after();
                if (idle) {
                    tc_fence_before();
                    mbar_arrive(bar(kSbP + x));
                    continue;
                }
                float s[kSpTile];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    tmem_ld32(lane_base + sp_col_s(x) + 32 * q, s + 32 * q);
                tmem_wait_ld();
                int lim = sg.g.pre_len - j * kSpTile;   // keys of the tile that exist
                if constexpr (kWhole) {
                    if (j >= sg.g.nt) {   // that the row sees: none of another request's
                        const DevShared &rq = reqs[ot.b];
                        const int t = tok - rq.q_off;
                        lim = t >= 0 && t < rq.q_len ? rq.own + t + 1 - ot.k * kSpTile : 0;
                        ot.next(reqs, sa->n_reqs);
                    }
                }
                if (lim < kSpTile) {
#pragma unroll
                    for (int c = 0; c < kSpTile; ++c)
                        s[c] = (c < lim) ? s[c] : -INFINITY;
                }
                float m4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int c = 4; c + 4 < kSpTile; c += 8) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        m4[k] = max3(m4[k], s[c + 2 * k], s[c + 2 * k + 1]);
                }
                const float mxs = max3(max3(m4[0], m4[1], m4[2]), m4[3],
                                       max3(max3(s[kSpTile - 4], s[kSpTile - 3], s[kSpTile - 2]), s[kSpTile - 1], m4[0])) * sc;
                // lazy maximum: O and l are rescaled only when it grows by more than
                // the threshold
                float corr = 1.f;
                if (j == sg.jb) {
                    m_run = mxs;
                } else if (mxs > m_run + kSpRescale) {
                    corr = ex2(m_run - mxs);
                    m_run = mxs;
                }
                // (all lanes together: tcgen05 loads and stores under a lane's own
                // condition may never return)
                const bool rescale = __any_sync(0xffffffffu, corr != 1.f);
                const float nm = m_run == -INFINITY ? 0.f : -m_run;   // (a score of -inf in every key)
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
                    tmem_st16(lane_base + sp_col_s(x) + 16 * q, pk);
                }
                {
                    float a0, a1, b0, b1;
                    unpk2(acc[0], a0, a1);
                    unpk2(acc[1], b0, b1);
                    l_run = l_run * corr + ((a0 + a1) + (b0 + b1));
                }
                if (rescale) {
                    // the commit that signalled this S covers the P V before it: O is stable
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float o[32];
                        tmem_ld32(lane_base + sp_col_o(x) + 32 * q, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] *= corr;
                        tmem_st32(lane_base + sp_col_o(x) + 32 * q, o);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(bar(kSbP + x));
            }
            if (!ok)
                break;
            // the partial result: O (relative to m), m, l
            const int64_t slot = sg.item + blockIdx.x;
            if (!kWhole && row_ok)
                part_ml(a.part, slot, x)[r] = make_float2(m_run, l_run);
            if (!mbar_wait_warp(bar(kSbO + x), (uint32_t)o_cnt & 1, abort_flag)) {
                ok = false;
                break;
            }
            ++o_cnt;
            tc_fence_after();
            if constexpr (kWhole) {   // the row's output
                const int lh = a.lh_base + sg.lh, l = lh / sa->n_kv_heads, h = lh - l * sa->n_kv_heads;
                const int g = sg.row0 + x * 128 + r - (tok - sg.g.q_off) * a.group;
                uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(sa->out) +
                                                       (((int64_t)l * a.total_q + tok) * sa->n_q_heads + h * a.group + g) * kSpD);
                const float inv = 1.f / l_run;
                if (row_ok && !(l_run > 0.f && l_run < INFINITY))
                    atomicCAS(a.err, kDevOk, kDevBadInput);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float o[32];
                    tmem_ld32(lane_base + sp_col_o(x) + 32 * q, o);
                    tmem_wait_ld();
                    if (row_ok) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            dst[4 * q + i] = make_uint4(pack_bf16(o[8 * i] * inv, o[8 * i + 1] * inv),
                                                        pack_bf16(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                                                        pack_bf16(o[8 * i + 4] * inv, o[8 * i + 5] * inv),
                                                        pack_bf16(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
                    }
                }
                tc_fence_before();
                mbar_arrive(bar(kSbOEmpty + x));
                continue;
            }
            float4 *po = part_o(a.part, slot, x) + r;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float o[32];
                tmem_ld32(lane_base + sp_col_o(x) + 32 * q, o);
                tmem_wait_ld();
                if (row_ok) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        po[(8 * q + i) * 128] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                }
            }
            tc_fence_before();
            mbar_arrive(bar(kSbOEmpty + x));
        }
        if (!ok)
            give_up(a.err, abort_flag);
    } else if (warp == 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kSpRegsOther));
        if (lane == 0) {
            // The kernel before (the prologue) does not write the prefix: once it passed on
            // that what came before the call is done, the first tiles, and the tables, are
            // read ahead of the wait for it; the packed queries are not.
            bool ok = true, waited = !relay_seen(a.relay, a.call);
            if (waited)
                pdl_wait_prerequisites();
            int tt = 0, nq = 0;
            for (int64_t w = w_begin; w < w_end && ok;) {
                OwnTiles ot;
                const Seg sg = seg(w, ot);
                w = sg.next;
                const int64_t kv0 = sg.g.pre_row0 + (int64_t)(a.lh_base + sg.lh) * sg.g.pre_cap;
                const int n_loads = 2 * (sg.je - sg.jb);
                for (int i = 0; i <= n_loads && ok; ++i) {
                    if (i == 2) {   // the queries after the first K and V tile
                        if (!waited) {
                            pdl_wait_prerequisites();
                            waited = true;
                        }
                        if (nq > 0 && !mbar_wait(bar(kSbQEmpty), (uint32_t)(nq - 1) & 1, abort_flag)) {
                            ok = false;
                            break;
                        }
                        const int q0 = (int)(((int64_t)(a.lh_base + sg.lh) * a.total_q + sg.g.q_off) * a.group + sg.row0);
                        mbar_expect_tx(bar(kSbQ), (uint32_t)(sg.nx * kSpTileBytes));
                        for (int x = 0; x < sg.nx; ++x) {
                            const uint32_t dst = sbase + (uint32_t)(kSpOffQ + x * kSpTileBytes);
                            tma_load_2d(dst, &tmq, 0, q0 + x * kSpTile, bar(kSbQ));
                            tma_load_2d(dst + kSpPanel, &tmq, 64, q0 + x * kSpTile, bar(kSbQ));
                        }
                        ++nq;
                    }
                    if (i == n_loads)
                        break;
                    const int slot = tt % kSpSlots;
                    if (tt >= kSpSlots && !mbar_wait(bar(kSbEmpty + slot), (uint32_t)(tt / kSpSlots - 1) & 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = sbase + (uint32_t)(kSpOffKV + slot * kSpTileBytes);
                    const CUtensorMap *map = (i & 1) ? &tmv : &tmk;
                    int row = (int)(kv0 + (int64_t)(sg.jb + (i >> 1)) * kSpTile);
                    if constexpr (kWhole) {
                        if ((i >> 1) >= sg.g.nt) {
                            const DevShared &rq = reqs[ot.b];
                            map = (i & 1) ? &tmov : &tmok;
                            row = (int)(rq.cache_row0 + (int64_t)(a.lh_base + sg.lh) * rq.cap + ot.k * kSpTile);
                            if (i & 1)
                                ot.next(reqs, sa->n_reqs);
                        }
                    }
                    mbar_expect_tx(bar(kSbFull + slot), kSpTileBytes);
                    tma_load_2d(dst, map, 0, row, bar(kSbFull + slot));
                    tma_load_2d(dst + kSpPanel, map, 64, row, bar(kSbFull + slot));
                    ++tt;
                }
            }
            if (!ok)
                give_up(a.err, abort_flag);
            for (int k = tt > kSpSlots ? tt - kSpSlots : 0; k < tt; ++k)
                mbar_drain(bar(kSbFull + k % kSpSlots), (uint32_t)(k / kSpSlots) & 1);
            if (nq > 0)
                mbar_drain(bar(kSbQ), (uint32_t)(nq - 1) & 1);
        }
    } else if (warp == 9) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kSpRegsOther));
        pdl_wait_prerequisites();   // (it reads the tables)
        const uint32_t lead = elect_one();
        int tt = 0, nq = 0, p_cnt[2] = {0, 0}, oe_cnt[2] = {0, 0};
        bool o_used[2] = {false, false}, ok = true;
        const uint64_t d_k = sdesc(sbase, 16, 1024), d_v = sdesc(sbase, kSpPanel, 1024);
        const uint32_t lo_k = (uint32_t)d_k, hi_k = (uint32_t)(d_k >> 32), lo_v = (uint32_t)d_v, hi_v = (uint32_t)(d_v >> 32);
        auto wait_kv = [&](int k) -> bool {
            if (!mbar_wait_warp(bar(kSbFull + k % kSpSlots), (uint32_t)(k / kSpSlots) & 1, abort_flag))
                return false;
            tc_fence_after();
            return true;
        };
        // S_x = Q_x K^T with K the ring's load k
        auto issue_s = [&](int x, int k) {
            const uint32_t qa = lo_k + ((uint32_t)(kSpOffQ + x * kSpTileBytes) >> 4);
            const uint32_t kb = lo_k + ((uint32_t)(kSpOffKV + (k % kSpSlots) * kSpTileBytes) >> 4);
#pragma unroll
            for (int i = 0; i < kSpD / 16; ++i) {
                const uint32_t off = (uint32_t)((i >> 2) * kSpPanel + (i & 3) * 32) >> 4;
                mma_ss(lead, tmem + sp_col_s(x), desc_with_lo(qa + off, hi_k), desc_with_lo(kb + off, hi_k), kSpIdescS, i > 0);
            }
            umma_commit(lead, bar(kSbS + x));
        };
        auto issue_pv = [&](int x, int k, uint32_t acc0) {
            const uint32_t vb = lo_v + ((uint32_t)(kSpOffKV + (k % kSpSlots) * kSpTileBytes) >> 4);
#pragma unroll
            for (int i = 0; i < kSpTile / 16; ++i)
                mma_ts(lead, tmem + sp_col_o(x), tmem + sp_col_s(x) + 8 * i, desc_with_lo(vb + ((i * 2048) >> 4), hi_v),
                       kSpIdescPV, i > 0 ? 1u : acc0);
        };
        // An own tile's P V, for rows lo .. hi - 1 of tile x alone: another
        // request's rows have weights of 0, but 0 x NaN would reach them.
        auto issue_pv_rows = [&](int x, int k, int lo, int hi) {
            const uint32_t vb = lo_v + ((uint32_t)(kSpOffKV + (k % kSpSlots) * kSpTileBytes) >> 4);
            uint32_t off[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int a0 = min(32, max(0, lo - 32 * i)), a1 = min(32, max(0, hi - 32 * i));
                const uint32_t below_lo = a0 == 32 ? ~0u : (1u << a0) - 1u, below_hi = a1 == 32 ? ~0u : (1u << a1) - 1u;
                off[i] = ~(below_hi & ~below_lo);
            }
#pragma unroll
            for (int i = 0; i < kSpTile / 16; ++i)
                mma_ts_rows(lead, tmem + sp_col_o(x), tmem + sp_col_s(x) + 8 * i,
                            desc_with_lo(vb + ((i * 2048) >> 4), hi_v), kSpIdescPV, 1u, off);
        };
        for (int64_t w = w_begin; w < w_end && ok;) {
            OwnTiles ot;
            const Seg sg = seg(w, ot);
            w = sg.next;
            const int K = sg.je - sg.jb;
            // V tile i of the segment: landed, its rows behind the prefix zeroed
            auto wait_v = [&](int i) -> bool {
                if (!wait_kv(tt + 2 * i + 1))
                    return false;
                int lim = sg.g.pre_len - (sg.jb + i) * kSpTile;
                if constexpr (kWhole) {
                    if (i >= sg.g.nt) {
                        const DevShared &rq = reqs[ot.b];
                        lim = rq.own + rq.q_len - ot.k * kSpTile;
                    }
                }
                if (lim < kSpTile) {
                    const uint32_t v = sbase + (uint32_t)(kSpOffKV + ((tt + 2 * i + 1) % kSpSlots) * kSpTileBytes);
                    for (int c = lim * 8 + lane; c < kSpTile * 8; c += 32) {
                        st_shared_v4(v + 16u * (uint32_t)c, 0u, 0u, 0u, 0u);
                        st_shared_v4(v + kSpPanel + 16u * (uint32_t)c, 0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                return true;
            };
            auto o_free = [&](int x) -> bool {
                if (o_used[x]) {
                    if (!mbar_wait_warp(bar(kSbOEmpty + x), (uint32_t)oe_cnt[x] & 1, abort_flag))
                        return false;
                    ++oe_cnt[x];
                    o_used[x] = false;
                }
                return true;
            };
            if (!mbar_wait_warp(bar(kSbQ), (uint32_t)nq & 1, abort_flag)) {
                ok = false;
                break;
            }
            ++nq;
            tc_fence_after();
            // the first S of each tile
            ok = wait_kv(tt);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                ok = ok && (x >= sg.nx || o_free(x));
                if (ok && x < sg.nx)
                    issue_s(x, tt);
            }
            if (!ok)
                break;
            umma_commit(lead, bar(kSbEmpty + tt % kSpSlots));
            if (K == 1)
                umma_commit(lead, bar(kSbQEmpty));
            for (int i = 0; i < K && ok; ++i) {
                const bool more = i + 1 < K;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (x >= sg.nx)
                        break;
                    if (!mbar_wait_warp(bar(kSbP + x), (uint32_t)p_cnt[x] & 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    ++p_cnt[x];
                    if (x == 0 && !wait_v(i)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (kWhole && i >= sg.g.nt) {
                        const DevShared &rq = reqs[ot.b];
                        const int lo = (rq.q_off - sg.g.q_off) * a.group - sg.row0 - x * kSpTile;
                        issue_pv_rows(x, tt + 2 * i + 1, lo, lo + rq.q_len * a.group);
                    } else {
                        issue_pv(x, tt + 2 * i + 1, i > 0);
                    }
                    if (!more) {
                        umma_commit(lead, bar(kSbO + x));
                        o_used[x] = true;
                    } else {
                        if (x == 0 && !wait_kv(tt + 2 * i + 2)) {
                            ok = false;
                            break;
                        }
                        issue_s(x, tt + 2 * i + 2);
                    }
                }
                if (!ok)
                    break;
                if (kWhole && i >= sg.g.nt)
                    ot.next(reqs, sa->n_reqs);
                if (i + 2 == K)
                    umma_commit(lead, bar(kSbQEmpty));   // the segment's last S is issued
                umma_commit(lead, bar(kSbEmpty + (tt + 2 * i + 1) % kSpSlots));
                if (more)
                    umma_commit(lead, bar(kSbEmpty + (tt + 2 * i + 2) % kSpSlots));
            }
            tt += 2 * K;
        }
        if (!ok)
            give_up(a.err, abort_flag);
        umma_commit(lead, bar(kSbDrain));
        mbar_drain(bar(kSbDrain), 0);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kSpRegsOther));
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, kSpTmemCols);
    }
}

}  // namespace

__global__ void __launch_bounds__(kSpThreads, 1)
    k_shared_prefix(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                    const __grid_constant__ CUtensorMap tmv, const __grid_constant__ SharedPrefixArgs a,
                    const __grid_constant__ GroupTable gt)
{
    prefix_part<false>(tmq, tmk, tmv, a, a.groups ? a.groups : gt.groups, tmk, tmv, nullptr, nullptr);
}

__global__ void __launch_bounds__(kSpThreads, 1)
    k_shared_whole(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                   const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmok,
                   const __grid_constant__ CUtensorMap tmov, const __grid_constant__ SharedPrefixArgs a,
                   const __grid_constant__ GroupTable gt, const __grid_constant__ SharedArgs sa,
                   const __grid_constant__ SharedTable rt)
{
    prefix_part<true>(tmq, tmk, tmv, a, a.groups ? a.groups : gt.groups, tmok, tmov, &sa, sa.reqs ? sa.reqs : rt.reqs);
}

// ---------------------------------------------------------------------------
// the query side
// ---------------------------------------------------------------------------
namespace {
constexpr int kPrPairs = 16;                // (layer, token, kv-head) triples per CTA
constexpr int kPrThreads = 8 * kPrPairs;    // 8 threads each: elements [8j, 8j + 8) and [64 + 8j, ..)

__device__ __forceinline__ void rotate_row(uint4 &lo, uint4 &hi, const float *c, const float *s, bool il)
{
    if (il)
        rotate_bf16x8_il(lo, hi, c, s);
    else
        rotate_bf16x8(lo, hi, c, s);
}
}  // namespace

// One CTA: kPrPairs consecutive (layer, token, kv-head) triples of the call, in the
// order of the query tensor, so that the grid is the call's work whatever its requests'
// lengths (with a grid of requests x the longest one's triples, 64 requests, one of 2,048
// tokens, on 288 units took 19.4 ms a call; 17.0 with this one).
__global__ void __launch_bounds__(kPrThreads)
    k_shared_prologue(const __grid_constant__ SharedArgs a, const __grid_constant__ SharedTable rt,
                      __nv_bfloat16 *__restrict__ q_rot)
{
    constexpr int D = kSpD, H2 = D / 2, E = 8;
    const DevShared *reqs = a.reqs ? a.reqs : rt.reqs;
    pdl_wait_prerequisites();
    if (blockIdx.x == 0 && threadIdx.x == 0)
        relay_store(a.relay, a.call);
    pdl_launch_dependents();   // the attention kernel sets up, and loads prefix tiles, meanwhile
    const int H = a.n_kv_heads, G = a.n_q_heads / H;
    const unsigned i = blockIdx.x * (unsigned)kPrPairs + (threadIdx.x >> 3);   // (L T Hq < 2^31)
    const int j = threadIdx.x & 7;
    if (i >= (unsigned)a.n_layers * (unsigned)a.total_q * (unsigned)H)
        return;
    const int h = (int)(i % (unsigned)H), lt = (int)(i / (unsigned)H), l = lt / a.total_q, t_all = lt - l * a.total_q;
    const int lh = l * H + h;
    const int64_t T = a.total_q, tok = lt;
    const __nv_bfloat16 *__restrict__ q = static_cast<const __nv_bfloat16 *>(a.q);
    const __nv_bfloat16 *__restrict__ kq = static_cast<const __nv_bfloat16 *>(a.kq);
    const __nv_bfloat16 *__restrict__ vq = static_cast<const __nv_bfloat16 *>(a.vq);
    __nv_bfloat16 *ck = static_cast<__nv_bfloat16 *>(a.cache_k), *cv = static_cast<__nv_bfloat16 *>(a.cache_v);
    const int64_t src = (tok * H + h) * D + j * E;
    uint4 klo = *reinterpret_cast<const uint4 *>(kq + src), khi = *reinterpret_cast<const uint4 *>(kq + src + H2);
    const uint4 vlo = *reinterpret_cast<const uint4 *>(vq + src), vhi = *reinterpret_cast<const uint4 *>(vq + src + H2);
    // the token's request: the last one that starts at or before it; where requests are as
    // long as one another (a decode step), the one that it would be then
    int b = min((int)(((float)t_all + 0.5f) * __fdividef((float)a.n_reqs, (float)a.total_q)), a.n_reqs - 1);
    if (reqs[b].q_off > t_all || reqs[b].q_off + reqs[b].q_len <= t_all) {
        int last = a.n_reqs - 1;
        b = 0;
        while (b < last) {
            const int mid = (b + last + 1) >> 1;
            if (reqs[mid].q_off <= t_all)
                b = mid;
            else
                last = mid - 1;
        }
    }
    const DevShared &rq = reqs[b];
    const int t = t_all - rq.q_off;
    float c[E], s[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const float2 cs = rope_cs(a.rope, H2, rq.pre_len + rq.own + t, rope_pair(a.interleaved, D, E, j, e));
        c[e] = cs.x;
        s[e] = cs.y;
    }
    const int64_t q_src = (tok * a.n_q_heads + (int64_t)h * G) * D + j * E;
    const int64_t q_dst = ((int64_t)lh * T + t_all) * G * D + j * E;
#pragma unroll 4
    for (int g = 0; g < G; ++g) {
        uint4 lo = *reinterpret_cast<const uint4 *>(q + q_src + (int64_t)g * D);
        uint4 hi = *reinterpret_cast<const uint4 *>(q + q_src + (int64_t)g * D + H2);
        rotate_row(lo, hi, c, s, a.interleaved);
        *reinterpret_cast<uint4 *>(q_rot + q_dst + (int64_t)g * D) = lo;
        *reinterpret_cast<uint4 *>(q_rot + q_dst + (int64_t)g * D + H2) = hi;
    }
    rotate_row(klo, khi, c, s, a.interleaved);
    const int64_t dst = (rq.cache_row0 + (int64_t)lh * rq.cap + rq.own + t) * D + j * E;
    *reinterpret_cast<uint4 *>(ck + dst) = klo;
    *reinterpret_cast<uint4 *>(ck + dst + H2) = khi;
    *reinterpret_cast<uint4 *>(cv + dst) = vlo;
    *reinterpret_cast<uint4 *>(cv + dst + H2) = vhi;
}

// ---------------------------------------------------------------------------
// the own part and the sum
// ---------------------------------------------------------------------------
namespace {
constexpr int kOwThreads = 128;
constexpr int kOwRowsMax = kOwnRowsMax;
constexpr int kOwTileMax = 128;   // keys per tile
// Shared memory of k_shared_own_rows: K and V tile ([tile_keys][128], two
// 128B-swizzled panels each), the barrier.
__host__ __device__ constexpr int ow_bytes(int tile_keys) { return tile_keys * 512 + 16 + 1024; }

// Where the partial results of one row lie: slots [slot, slot + n), row `in` of
// each (of its two tiles).
struct PartRef {
    int64_t slot;
    int n, in;
};

__device__ __forceinline__ PartRef part_ref(const SharedPrefixArgs &pa, const DevGroup &g, int lh_s, int group_row)
{
    PartRef r{0, 0, 0};
    if (g.nt == 0)
        return r;
    const int blk = group_row >> 8;
    const int64_t it = (int64_t)lh_s * pa.unit_blocks + g.item0 + blk;
    const int64_t w0 = (int64_t)lh_s * pa.unit_pairs + g.w0 + (int64_t)blk * g.nt;
    const int ca = stretch_of(pa.total, pa.n_ctas, pa.ratio, w0);
    const int cb = stretch_of(pa.total, pa.n_ctas, pa.ratio, w0 + g.nt - 1);
    r.slot = it + ca;
    r.n = cb - ca + 1;
    r.in = group_row & 255;
    return r;
}

// Bounded wait that reads the timer only when the phase is not complete yet (a
// %globaltimer read costs some 600 cycles).
__device__ __forceinline__ bool own_wait(uint32_t bar, uint32_t parity)
{
    return mbar_try_wait(bar, parity) || mbar_drain(bar, parity);
}

// What the end of a row tile needs to know of the prefix's partial results of
// its rows (NH: row r_first, and r_first + 8 too), looked up ahead of the row
// tile's work.
struct RowParts {
    PartRef pr[2];
    float2 v[2][2];   // (max, sum) of the first two partial results (none: -inf, 0)

    __device__ __forceinline__ int n(int hh) const { return pr[hh].n; }
    __device__ __forceinline__ float2 ml(const SharedPrefixArgs &pa, int hh, int i) const
    {
        return part_ml(pa.part, pr[hh].slot + i, pr[hh].in >> 7)[pr[hh].in & 127];
    }
    // columns cq, cq + 1 of partial result i; the next 8 columns are 1024 floats on
    __device__ __forceinline__ const float *o(const SharedPrefixArgs &pa, int hh, int i, int cq) const
    {
        return reinterpret_cast<const float *>(part_o(pa.part, pr[hh].slot + i, pr[hh].in >> 7) + (cq >> 2) * 128 +
                                               (pr[hh].in & 127)) + (cq & 3);
    }
};
template <int NH>
__device__ __forceinline__ RowParts row_parts(const SharedPrefixArgs &pa, const DevGroup &g, const DevShared &rq, int lh_s,
                                              int r_first, int m_rows)
{
    RowParts p;
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
        const int r = r_first + 8 * hh;
        p.pr[hh] = PartRef{0, 0, 0};
        if (hh < NH && r < m_rows)
            p.pr[hh] = part_ref(pa, g, lh_s, (rq.q_off - g.q_off) * pa.group + r);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            p.v[hh][i] = hh < NH && i < p.n(hh) ? p.ml(pa, hh, i) : make_float2(-INFINITY, 0.f);
    }
    return p;
}

// The O of the first two partial results of a row tile's first row half, in
// registers ahead of their use.
struct EarlyO {
    float2 f[2][16];
    __device__ __forceinline__ void load(const SharedPrefixArgs &pa, const RowParts &rp, int cq)
    {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            // (a result whose sum is 0 has an undefined O: read, where it exists, and not used)
            const float *po = i < rp.n(0) ? rp.o(pa, 0, i, cq) : nullptr;
#pragma unroll
            for (int nn = 0; nn < 16; ++nn)
                f[i][nn] = po ? *reinterpret_cast<const float2 *>(po + nn * 1024) : make_float2(0.f, 0.f);
        }
    }
};
struct NoEarlyO {};

// The end of a row tile: adds the prefix's partial results (in stretch order) to
// the warp's own states and writes the rows.  Lane: columns 8n + cq, + 1 of row
// r_first of the request and (NH 2) of row r_first + 8 (fragment layout); l_run
// holds the lane's keys only.
template <int NH, typename Early>
__device__ __forceinline__ void finish_rows(const SharedArgs &a, const SharedPrefixArgs &pa, const RowParts &rp,
                                            const Early &early, const DevShared &rq, int lh_s, int r_first, int m_rows,
                                            float (&o)[16][4], const float *m_run, const float *l_run)
{
    constexpr bool kEarly = !std::is_same<Early, NoEarlyO>::value;
    const int lane = threadIdx.x & 31, cq = (lane & 3) * 2, G = pa.group;
    const int lh = pa.lh_base + lh_s, l = lh / a.n_kv_heads, h = lh - l * a.n_kv_heads;
#pragma unroll
    for (int hh = 0; hh < NH; ++hh) {
        const int r = r_first + 8 * hh, n = rp.n(hh);
        float L = l_run[hh];
        L += __shfl_xor_sync(0xffffffffu, L, 1);
        L += __shfl_xor_sync(0xffffffffu, L, 2);
        if (r >= m_rows)
            continue;
        auto state = [&](int i) -> float2 { return i < 2 ? rp.v[hh][i] : rp.ml(pa, hh, i); };
        float M = L == 0.f ? -INFINITY : m_run[hh];   // (a sum of 0: no key counts)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            M = rp.v[hh][i].y == 0.f ? M : fmaxf(M, rp.v[hh][i].x);
        for (int i = 2; i < n; ++i) {
            const float2 v = state(i);
            M = v.y == 0.f ? M : fmaxf(M, v.x);
        }
        const float w_own = L == 0.f ? 0.f : dec::dec_ex2(m_run[hh] - M);
        L *= w_own;
#pragma unroll
        for (int nn = 0; nn < 16; ++nn) {
            o[nn][2 * hh] *= w_own;
            o[nn][2 * hh + 1] *= w_own;
        }
        auto add = [&](float2 v, const float2 (&f)[16]) {
            const float wt = dec::dec_ex2(v.x - M);
            L += v.y * wt;
#pragma unroll
            for (int nn = 0; nn < 16; ++nn) {
                o[nn][2 * hh] = fmaf(f[nn].x, wt, o[nn][2 * hh]);
                o[nn][2 * hh + 1] = fmaf(f[nn].y, wt, o[nn][2 * hh + 1]);
            }
        };
        int i = 0;
        if constexpr (kEarly) {
            if (hh == 0) {
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    if (rp.v[0][x].y != 0.f)
                        add(rp.v[0][x], early.f[x]);
                i = 2;
            }
        }
        for (; i < n; ++i) {
            const float2 v = state(i);
            if (v.y == 0.f)   // (its O is undefined)
                continue;
            const float *po = rp.o(pa, hh, i, cq);
            float2 f[16];
#pragma unroll
            for (int nn = 0; nn < 16; ++nn)
                f[nn] = *reinterpret_cast<const float2 *>(po + nn * 1024);
            add(v, f);
        }
        if ((lane & 3) == 0 && !(L > 0.f && L < INFINITY))
            atomicCAS(a.err, kDevOk, kDevBadInput);
        const float inv = 1.f / L;
        const int tk = r / G;
        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.out) +
                             (((int64_t)l * a.total_q + rq.q_off + tk) * a.n_q_heads + h * G + (r - tk * G)) * kSpD + cq;
#pragma unroll
        for (int nn = 0; nn < 16; ++nn)
            *reinterpret_cast<uint32_t *>(dst + 8 * nn) = dec::pack2(o[nn][2 * hh] * inv, o[nn][2 * hh + 1] * inv);
    }
}
}  // namespace

// More than 16 query rows a request (an MMA row tile of the kernel below): a CTA
// takes `tiles_per_cta` groups of 64 rows of a (request, unit); each warp has a
// row tile of its own and takes all keys of a tile.  Own parts of one tile are
// loaded once per CTA, and its warps then go through their rows independently.
// Bound by the reads of queries and partial results: 708,736 rows of 49 to 64
// keys: 225 us, 3.5 TB/s.  (With 4 rows a request, three of four warps are idle: a
// step of 64 requests on 8,256 rows takes 491 us with it, 391 with the kernel
// below.)
__global__ void __launch_bounds__(kOwThreads, 3)
    k_shared_own_rows(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                 const __grid_constant__ SharedArgs a, const __grid_constant__ SharedTable rt,
                 const __grid_constant__ SharedPrefixArgs pa, const __grid_constant__ GroupTable gt, const int tiles_per_cta,
                 const int tile_keys)
{
    using namespace dec;
    extern __shared__ uint8_t ow_smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(ow_smem_raw) + 1023) & ~uintptr_t(1023));
    const int panel = tile_keys * 128, kOwTile = tile_keys, off_bar = 4 * panel;
    const uint32_t sbase = dec_smem_u32(smem), kt = sbase, vt = sbase + 2 * panel, full = sbase + off_bar;
    volatile int *cta_err = reinterpret_cast<volatile int *>(smem + off_bar + 8);
    auto sw = [&](int r, int c) { return (uint32_t)((c >> 3) * panel + r * 128 + (((c & 7) ^ (r & 7)) << 4)); };
    const DevShared *reqs = a.reqs ? a.reqs : rt.reqs;
    const DevGroup *groups = pa.groups ? pa.groups : gt.groups;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = pa.group;
    if (a.reqs)
        pdl_wait_prerequisites();   // (the table was uploaded)
    // this CTA's request: the last one whose first chunk is at or before the CTA's (those
    // behind it, without chunks, begin where the next one does); where requests have as many
    // chunks as one another, the one that it would be then
    const int rows_cta = tiles_per_cta * kOwRowsMax;
    auto chunks_of = [&](const DevShared &r) { return r.q_len * G > kOwnFewRows ? (r.q_len * G + rows_cta - 1) / rows_cta : 0; };
    int b = min((int)(((float)blockIdx.x + 0.5f) * __fdividef((float)a.n_reqs, (float)gridDim.x)), a.n_reqs - 1);
    if (reqs[b].chunk0 * pa.lh_count > (int)blockIdx.x || (reqs[b].chunk0 + chunks_of(reqs[b])) * pa.lh_count <= (int)blockIdx.x) {
        int last = a.n_reqs - 1;
        b = 0;
        while (b < last) {
            const int mid = (b + last + 1) >> 1;
            if (reqs[mid].chunk0 * pa.lh_count <= (int)blockIdx.x)
                b = mid;
            else
                last = mid - 1;
        }
    }
    const DevShared rq = reqs[b];
    const int m_rows = rq.q_len * G, n_chunks = chunks_of(rq), in_req = (int)blockIdx.x - rq.chunk0 * pa.lh_count;
    const int lh_s = in_req / n_chunks, lh = pa.lh_base + lh_s, r_first = (in_req - lh_s * n_chunks) * rows_cta;
    const int r_last = min(m_rows, r_first + rows_cta);
    auto keys_to = [&](int r_end) { return rq.own + (r_end - 1) / G + 1; };   // keys of the rows before r_end
    const bool once = keys_to(r_last) <= kOwTile;
    const int64_t kv_row0 = rq.cache_row0 + (int64_t)lh * rq.cap;
    int n_keys = keys_to(once ? r_last : min(r_last, r_first + kOwRowsMax));

    auto issue = [&](int j) {   // thread 0
        const int n32 = min(kOwTile >> 5, (n_keys - j * kOwTile + 31) >> 5);
        dec_expect_tx(full, (uint32_t)(n32 * 32 * kSpD * 2 * 2));
        for (int i = 0; i < n32; ++i) {
            const int row = (int)(kv_row0 + (int64_t)j * kOwTile + 32 * i);
            const uint32_t d = (uint32_t)(i * 32 * 128);
            dec_tma_load(kt + d, &tmk, 0, row, full);
            dec_tma_load(kt + panel + d, &tmk, 64, row, full);
            dec_tma_load(vt + d, &tmv, 0, row, full);
            dec_tma_load(vt + panel + d, &tmv, 64, row, full);
        }
    };
    if (threadIdx.x == 0) {
        dec_mbar_init(full, 1);
        *cta_err = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        pdl_wait_prerequisites();
        issue(0);
    } else {
        pdl_wait_prerequisites();
    }
    __syncthreads();   // the barrier is initialised
    const float sc = a.scale_log2;
    const int rt0 = 16 * warp;   // the warp's row tile in a group
    const int ra = rt0 + (lane >> 2), rb = ra + 8, cq = (lane & 3) * 2;
    int step = 0;   // tiles loaded
    for (int r0 = r_first; r0 < r_last; r0 += kOwRowsMax) {
        const int rows = min(kOwRowsMax, r_last - r0);
        if (!once && r0 > r_first) {
            n_keys = keys_to(r0 + rows);
            if (threadIdx.x == 0)
                issue(0);
        }
        const int n_t = (n_keys + kOwTile - 1) / kOwTile;
        // query fragments (A operand): rows ra, rb of this warp's row tile
        const __nv_bfloat16 *qp = static_cast<const __nv_bfloat16 *>(pa.q_rot) +
                                  (((int64_t)lh * a.total_q + rq.q_off) * G + r0) * kSpD;
        uint32_t qa[8][4];
#pragma unroll
        for (int kb = 0; kb < 8; ++kb) {
            const int c0 = kb * 16 + cq;
            auto ld2 = [&](int r, int c) -> uint32_t {
                return r < rows ? *reinterpret_cast<const uint32_t *>(qp + (int64_t)r * kSpD + c) : 0u;
            };
            qa[kb][0] = ld2(ra, c0);
            qa[kb][1] = ld2(rb, c0);
            qa[kb][2] = ld2(ra, c0 + 8);
            qa[kb][3] = ld2(rb, c0 + 8);
        }
        // keys that the two rows see
        const int see[2] = {ra < rows ? rq.own + (r0 + ra) / G + 1 : 0, rb < rows ? rq.own + (r0 + rb) / G + 1 : 0};
        const int see_warp = rt0 < rows ? rq.own + (r0 + min(rt0 + 15, rows - 1)) / G + 1 : 0;
        float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
        float o[16][4];
#pragma unroll
        for (int n = 0; n < 16; ++n)
            o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
        for (int j = 0; j < n_t; ++j) {
            const int kk0 = j * kOwTile, n_here = min(kOwTile, n_keys - kk0);
            if (!once || r0 == r_first) {
                if (!own_wait(full, (uint32_t)step & 1))
                    *cta_err = 1;
                // V rows behind the last key are zero (32-row groups that were loaded)
                const int n_ld = (n_here + 31) & ~31;
                for (int idx = threadIdx.x; idx < (n_ld - n_here) * 16; idx += kOwThreads)
                    st_shared_v4(vt + sw(n_here + (idx >> 4), idx & 15), 0u, 0u, 0u, 0u);
                fence_proxy_async_smem();   // (before the tile's next TMA write)
                __syncthreads();
                if (*cta_err) {   // the same for every thread
                    if (threadIdx.x == 0) {
                        atomicCAS(a.err, kDevOk, kDevTimeout);
                        mbar_drain(full, (uint32_t)step & 1);
                    }
                    return;
                }
                ++step;
            }
            const int n_warp = min(n_here, see_warp - kk0);   // keys that some row of the warp sees
            for (int key0 = 0; key0 < n_warp; key0 += 32) {
                float c[4][4];
#pragma unroll
                for (int nb = 0; nb < 4; ++nb)
                    c[nb][0] = c[nb][1] = c[nb][2] = c[nb][3] = 0.f;
#pragma unroll
                for (int nb = 0; nb < 4; nb += 2) {
#pragma unroll
                    for (int kb = 0; kb < 8; ++kb) {
                        const int mi = lane >> 3;
                        const int key = key0 + 8 * (nb + (mi >> 1)) + (lane & 7);
                        uint32_t b0, b1, b2, b3;
                        ldsm_x4(kt + sw(key, 2 * kb + (mi & 1)), b0, b1, b2, b3);
                        mma_bf16(c[nb], qa[kb], b0, b1);
                        mma_bf16(c[nb + 1], qa[kb], b2, b3);
                    }
                }
                float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int nb = 0; nb < 4; ++nb) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int kk = kk0 + key0 + 8 * nb + cq + (e & 1);
                        c[nb][e] = kk < see[e >> 1] ? c[nb][e] * sc : -INFINITY;
                        mx[e >> 1] = fmaxf(mx[e >> 1], c[nb][e]);
                    }
                }
                float corr[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
                    mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
                    const float m_new = fmaxf(m_run[h], mx[h]);
                    corr[h] = m_new == -INFINITY ? 1.f : dec_ex2(m_run[h] - m_new);
                    m_run[h] = m_new;
                }
                const float nm[2] = {m_run[0] == -INFINITY ? 0.f : -m_run[0], m_run[1] == -INFINITY ? 0.f : -m_run[1]};
                float sum[2] = {0.f, 0.f};
                uint32_t p[2][4];
#pragma unroll
                for (int nb = 0; nb < 4; ++nb) {
                    const float p0 = dec_ex2(c[nb][0] + nm[0]), p1 = dec_ex2(c[nb][1] + nm[0]);
                    const float p2 = dec_ex2(c[nb][2] + nm[1]), p3 = dec_ex2(c[nb][3] + nm[1]);
                    sum[0] += p0 + p1;
                    sum[1] += p2 + p3;
                    p[nb >> 1][(nb & 1) * 2 + 0] = pack2(p0, p1);
                    p[nb >> 1][(nb & 1) * 2 + 1] = pack2(p2, p3);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)   // (this lane's keys only)
                    l_run[h] = l_run[h] * corr[h] + sum[h];
                if (j > 0 || key0 > 0) {   // (nothing to rescale in the first block)
#pragma unroll
                    for (int n = 0; n < 16; ++n) {
                        o[n][0] *= corr[0];
                        o[n][1] *= corr[0];
                        o[n][2] *= corr[1];
                        o[n][3] *= corr[1];
                    }
                }
#pragma unroll
                for (int kb2 = 0; kb2 < 2; ++kb2) {
#pragma unroll
                    for (int n = 0; n < 16; n += 2) {
                        const int mi = lane >> 3;
                        const int key = key0 + 16 * kb2 + 8 * (mi & 1) + (lane & 7);
                        uint32_t b0, b1, b2, b3;
                        ldsm_x4_t(vt + sw(key, n + (mi >> 1)), b0, b1, b2, b3);
                        mma_bf16(o[n], p[kb2], b0, b1);
                        mma_bf16(o[n + 1], p[kb2], b2, b3);
                    }
                }
            }
            if (!once) {
                __syncthreads();   // the tile is consumed
                if (threadIdx.x == 0 && j + 1 < n_t)
                    issue(j + 1);
            }
        }

        const RowParts parts = row_parts<2>(pa, groups[rq.group], rq, lh_s, r0 + ra, r0 + rows);
        finish_rows<2>(a, pa, parts, NoEarlyO{}, rq, lh_s, r0 + ra, r0 + rows, o, m_run, l_run);
    }
}

// At most 16 query rows a request (a decode step): the own rows are a stream of
// short pieces, one per (request, unit), and a piece's work is a chain of short
// dependent steps.  So every warp works by itself, on a consecutive stretch of
// pieces: its lane 0 loads the K and V rows 32 keys at a time, two steps ahead
// (across pieces), the warp runs S, softmax and P V of a step in registers, adds
// the prefix's partial results at the end of a piece and writes its rows.  Seven
// warps per SM, 32 KB of tiles each.  64 requests of 32 to 128 rows, 288 units:
// 166 us, 4.6 TB/s of K and V (a CTA a piece took 291), bound by the chain of a
// piece's steps: loads, three steps on average, partial results, output.  More
// warps have fewer registers: twelve, 16 KB each, without the early loads of the
// partial results, make the call 409 us instead of 394.  With at most 8 query
// rows the upper half of the MMA row tile is left out: 391 us a call against 400.
namespace {
constexpr int kOdWarps = 7;
constexpr int kOdThreads = 32 * kOdWarps;
constexpr int kOdTile = 32;
constexpr int kOdPanel = kOdTile * 128;           // 32 keys x 64 dims
constexpr int kOdStage = 4 * kOdPanel;            // K, then V: two panels each
constexpr int kOdOffBar = kOdWarps * 2 * kOdStage;
constexpr int kOdSmem = kOdOffBar + kOdWarps * 2 * 8 + 1024;   // + alignment slack

// 16-byte chunk c of row r of a tile
__device__ __forceinline__ uint32_t od_off(int r, int c)
{
    return (uint32_t)((c >> 3) * kOdPanel + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}
}  // namespace

// kTwo: more than 8 query rows (both halves of an MMA row tile hold some)
template <bool kTwo>
__global__ void __launch_bounds__(kOdThreads, 1)
    k_shared_own_decode(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                        const __grid_constant__ SharedArgs a, const __grid_constant__ SharedTable rt,
                        const __grid_constant__ SharedPrefixArgs pa, const __grid_constant__ GroupTable gt)
{
    using namespace dec;
    extern __shared__ uint8_t od_smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(od_smem_raw) + 1023) & ~uintptr_t(1023));
    const DevShared *reqs = a.reqs ? a.reqs : rt.reqs;
    const DevGroup *groups = pa.groups ? pa.groups : gt.groups;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t tiles = dec_smem_u32(smem) + (uint32_t)(warp * 2 * kOdStage);
    const uint32_t full0 = dec_smem_u32(smem) + (uint32_t)(kOdOffBar + warp * 16);
    const int G = pa.group, n_items = a.n_reqs * pa.lh_count;
    // the pieces of this warp; neighbours go to different SMs when there are few
    const int n_w = (int)gridDim.x * kOdWarps, w = warp * (int)gridDim.x + (int)blockIdx.x;
    const int it0 = (int)((int64_t)n_items * w / n_w), it1 = (int)((int64_t)n_items * (w + 1) / n_w);

    if (lane == 0) {
        dec_mbar_init(full0, 1);
        dec_mbar_init(full0 + 8, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_tmap(&tmk);
        prefetch_tmap(&tmv);
    }
    __syncwarp();
    // Behind a prefix part that passed on that the prologue is done, only the partial
    // results have to be waited for.
    bool waited = pa.total == 0;
    if (!waited) {
        waited = lane == 0 && !relay_seen(pa.relay + 1, pa.call);
        waited = __shfl_sync(0xffffffffu, waited, 0);
    }
    if (waited)
        pdl_wait_prerequisites();

    // (longer queries are k_shared_own_rows')
    auto takes = [&](const DevShared &r) { return r.q_len > 0 && r.q_len * G <= kOwnFewRows; };
    // the next step to load: tile `lj` of piece `li`
    int li = it0, lj = 0, l_keys = 0, n_issued = 0;
    int64_t l_row0 = 0;
    auto load_piece = [&]() {   // the first piece from li on with keys to load
        for (; li < it1; ++li) {
            const DevShared &r = reqs[li / pa.lh_count];
            if (takes(r)) {
                l_keys = r.own + r.q_len;
                l_row0 = r.cache_row0 + (int64_t)(pa.lh_base + li % pa.lh_count) * r.cap;
                return;
            }
        }
    };
    load_piece();
    auto issue = [&]() {
        if (li >= it1)
            return;
        if (lane == 0) {
            const uint32_t bar = full0 + 8u * (uint32_t)(n_issued & 1), dst = tiles + (uint32_t)((n_issued & 1) * kOdStage);
            const int row = (int)(l_row0 + (int64_t)lj * kOdTile);
            dec_expect_tx(bar, kOdStage);
            dec_tma_load(dst, &tmk, 0, row, bar);
            dec_tma_load(dst + kOdPanel, &tmk, 64, row, bar);
            dec_tma_load(dst + 2 * kOdPanel, &tmv, 0, row, bar);
            dec_tma_load(dst + 3 * kOdPanel, &tmv, 64, row, bar);
        }
        ++n_issued;
        if (++lj * kOdTile >= l_keys) {
            ++li;
            lj = 0;
            load_piece();
        }
    };
    issue();
    issue();

    // rows ra, rb and columns cq, cq + 1 (+ 8) of the MMA fragments
    constexpr int NH = kTwo ? 2 : 1;   // row halves with rows in them
    const int ra = lane >> 2, rb = ra + 8, cq = (lane & 3) * 2, mi = lane >> 3;
    const float sc = a.scale_log2;
    // the piece `it`, its packed queries as the MMA's A operand
    DevShared rq{};
    uint32_t qa[8][4];
    auto load_queries = [&](int it) {
        rq = reqs[it / pa.lh_count];
        const int m_rows = rq.q_len * G, lh = pa.lh_base + it % pa.lh_count;
        const __nv_bfloat16 *qp = static_cast<const __nv_bfloat16 *>(pa.q_rot) + ((int64_t)lh * a.total_q + rq.q_off) * G * kSpD;
#pragma unroll
        for (int kb = 0; kb < 8; ++kb) {
            auto ld2 = [&](int r, int c) -> uint32_t {
                return r < m_rows ? *reinterpret_cast<const uint32_t *>(qp + r * kSpD + c) : 0u;
            };
            qa[kb][0] = ld2(ra, kb * 16 + cq);
            qa[kb][1] = kTwo ? ld2(rb, kb * 16 + cq) : 0u;
            qa[kb][2] = ld2(ra, kb * 16 + cq + 8);
            qa[kb][3] = kTwo ? ld2(rb, kb * 16 + cq + 8) : 0u;
        }
    };
    if (it0 < it1)
        load_queries(it0);
    if (!waited)   // for the prefix's partial results
        pdl_wait_prerequisites();
    int k = 0;   // steps done
    bool ok = true;
    for (int it = it0; it < it1 && ok; ++it) {
        if (!takes(rq)) {
            if (it + 1 < it1)
                load_queries(it + 1);
            continue;
        }
        const DevShared req = rq;
        const int lh_s = it % pa.lh_count, m_rows = req.q_len * G;
        const int n_keys = req.own + req.q_len, n_t = (n_keys + kOdTile - 1) / kOdTile;
        const int see[2] = {ra < m_rows ? req.own + ra / G + 1 : 0, rb < m_rows ? req.own + rb / G + 1 : 0};
        // the first two partial results of the rows are on their way meanwhile
        const RowParts parts = row_parts<NH>(pa, groups[req.group], req, lh_s, ra, m_rows);
        EarlyO early;
        early.load(pa, parts, cq);
        float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
        float o[16][4];
#pragma unroll
        for (int n = 0; n < 16; ++n)
            o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
        for (int j = 0; j < n_t; ++j, ++k) {
            const uint32_t kt = tiles + (uint32_t)((k & 1) * kOdStage), vt = kt + 2 * kOdPanel;
            ok = own_wait(full0 + 8u * (uint32_t)(k & 1), (uint32_t)(k >> 1) & 1);
            if (!(ok = __all_sync(0xffffffffu, ok)))
                break;
            const int n_here = n_keys - j * kOdTile;
            if (n_here < kOdTile) {   // V rows behind the last key are zero
                for (int idx = lane; idx < (kOdTile - n_here) * 16; idx += 32)
                    st_shared_v4(vt + od_off(n_here + (idx >> 4), idx & 15), 0u, 0u, 0u, 0u);
                __syncwarp();
            }
            float c[4][4];
#pragma unroll
            for (int nb = 0; nb < 4; ++nb)
                c[nb][0] = c[nb][1] = c[nb][2] = c[nb][3] = 0.f;
#pragma unroll
            for (int kb = 0; kb < 8; ++kb) {
#pragma unroll
                for (int nb = 0; nb < 4; nb += 2) {
                    uint32_t b0, b1, b2, b3;
                    ldsm_x4(kt + od_off(8 * (nb + (mi >> 1)) + (lane & 7), 2 * kb + (mi & 1)), b0, b1, b2, b3);
                    mma_bf16(c[nb], qa[kb], b0, b1);
                    mma_bf16(c[nb + 1], qa[kb], b2, b3);
                }
            }
            float corr[2], nm[2];
            uint32_t p[2][4];
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                float mx = -INFINITY;
#pragma unroll
                for (int nb = 0; nb < 4; ++nb)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int kk = j * kOdTile + 8 * nb + cq + e;
                        float &s = c[nb][2 * h + e];
                        s = kk < see[h] ? s * sc : -INFINITY;
                        mx = fmaxf(mx, s);
                    }
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float m_new = fmaxf(m_run[h], mx);
                corr[h] = m_new == -INFINITY ? 1.f : dec_ex2(m_run[h] - m_new);
                m_run[h] = m_new;
                nm[h] = m_new == -INFINITY ? 0.f : -m_new;
                float sum = 0.f;
#pragma unroll
                for (int nb = 0; nb < 4; ++nb) {
                    const float p0 = dec_ex2(c[nb][2 * h] + nm[h]), p1 = dec_ex2(c[nb][2 * h + 1] + nm[h]);
                    sum += p0 + p1;
                    p[nb >> 1][(nb & 1) * 2 + h] = pack2(p0, p1);
                }
                l_run[h] = l_run[h] * corr[h] + sum;   // (this lane's keys only: added up over the quad at the end)
            }
            if (!kTwo) {   // the other row half: no rows, no weights
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    p[x][1] = p[x][3] = 0u;
            }
            if (j > 0) {
#pragma unroll
                for (int n = 0; n < 16; ++n)
#pragma unroll
                    for (int h = 0; h < NH; ++h) {
                        o[n][2 * h] *= corr[h];
                        o[n][2 * h + 1] *= corr[h];
                    }
            }
#pragma unroll
            for (int kb2 = 0; kb2 < 2; ++kb2) {
#pragma unroll
                for (int n = 0; n < 16; n += 2) {
                    uint32_t b0, b1, b2, b3;
                    ldsm_x4_t(vt + od_off(16 * kb2 + 8 * (mi & 1) + (lane & 7), n + (mi >> 1)), b0, b1, b2, b3);
                    mma_bf16(o[n], p[kb2], b0, b1);
                    mma_bf16(o[n + 1], p[kb2], b2, b3);
                }
            }
            if (n_here < kOdTile)
                fence_proxy_async_smem();   // the zeroed rows, before the stage's next TMA write
            __syncwarp();
            issue();
        }
        if (!ok)
            break;
        if (it + 1 < it1)
            load_queries(it + 1);   // on their way during the end of this piece
        finish_rows<NH>(a, pa, parts, early, req, lh_s, ra, m_rows, o, m_run, l_run);
        __syncwarp();
    }
    if (!ok) {   // nothing is in flight when the CTA leaves
        for (int x = k; x < n_issued; ++x)
            mbar_drain(full0 + 8u * (uint32_t)(x & 1), (uint32_t)(x >> 1) & 1);
        if (lane == 0)
            atomicCAS(a.err, kDevOk, kDevTimeout);
    }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
static cudaError_t shared_attrs()
{
    static std::atomic<bool> done[64] = {};   // per device (host threads may race: same values)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && done[dev].load(std::memory_order_acquire)))
        return e;
    // the register split must fit what the CTA is launched with, or the
    // softmax warpgroups' increase would wait forever
    cudaFuncAttributes fa{}, fw{};
    if ((e = cudaFuncGetAttributes(&fa, k_shared_prefix)) != cudaSuccess ||
        (e = cudaFuncGetAttributes(&fw, k_shared_whole)) != cudaSuccess)
        return e;
    if (fa.numRegs != kSpRegsLaunch || fw.numRegs != kSpRegsLaunch)
        return cudaErrorInvalidConfiguration;
    if ((e = cudaFuncSetAttribute(k_shared_prefix, cudaFuncAttributeMaxDynamicSharedMemorySize, kSpSmem)) != cudaSuccess ||
        (e = cudaFuncSetAttribute(k_shared_whole, cudaFuncAttributeMaxDynamicSharedMemorySize, kSpSmem)) != cudaSuccess ||
        (e = cudaFuncSetAttribute(k_shared_own_rows, cudaFuncAttributeMaxDynamicSharedMemorySize, ow_bytes(kOwTileMax))) !=
            cudaSuccess ||
        (e = cudaFuncSetAttribute(k_shared_own_decode<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kOdSmem)) !=
            cudaSuccess ||
        (e = cudaFuncSetAttribute(k_shared_own_decode<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kOdSmem)) != cudaSuccess)
        return e;
    if (dev < 64)
        done[dev].store(true, std::memory_order_release);
    return cudaSuccess;
}

cudaError_t launch_shared_prologue(const SharedArgs &a, const SharedTable &rt, void *q_rot, bool pdl, cudaStream_t s)
{
    const int64_t triples = (int64_t)a.n_layers * a.total_q * a.n_kv_heads;
    return launch_pdl(k_shared_prologue, (triples + kPrPairs - 1) / kPrPairs, kPrThreads, 0, pdl, s, a, rt,
                      static_cast<__nv_bfloat16 *>(q_rot));
}

cudaError_t launch_shared_tc(const SharedTcArgs &t, bool pdl, cudaStream_t s)
{
    cudaError_t e = shared_attrs();
    if (e != cudaSuccess)
        return e;
    const SharedArgs &a = *t.base;
    const SharedPrefixArgs &pa = *t.prefix;
    static const CUtensorMap no_map{};
    auto map = [](const void *m) -> const CUtensorMap & { return m ? *static_cast<const CUtensorMap *>(m) : no_map; };
    if (t.whole)
        return launch_pdl(k_shared_whole, pa.n_ctas, kSpThreads, kSpSmem, pdl, s, map(t.tmap_q), map(t.tmap_pk),
                          map(t.tmap_pv), map(t.tmap_k), map(t.tmap_v), pa, *t.groups, a, *t.reqs);
    if (pa.total > 0) {
        e = launch_pdl(k_shared_prefix, pa.n_ctas, kSpThreads, kSpSmem, pdl, s, map(t.tmap_q), map(t.tmap_pk),
                       map(t.tmap_pv), pa, *t.groups);
        if (e != cudaSuccess)
            return e;
    }
    if (t.few_rows > 0) {
        const int64_t items = (int64_t)a.n_reqs * pa.lh_count;
        if (items > 0x7fffffff)
            return cudaErrorInvalidValue;
        e = launch_pdl(t.few_rows <= 8 ? k_shared_own_decode<false> : k_shared_own_decode<true>, std::min<int64_t>(items, t.n_sms),
                       kOdThreads, kOdSmem, pdl, s, map(t.tmap_k), map(t.tmap_v), a, *t.reqs, pa, *t.groups);
        if (e != cudaSuccess || t.own_chunks == 0)
            return e;
    }
    // tiles that just hold the longest own part, cut evenly (a smaller tile
    // leaves room for more CTAs per SM)
    const int n_tiles = (t.max_own_keys + kOwTileMax - 1) / kOwTileMax;
    const int tile_keys = ((t.max_own_keys + n_tiles - 1) / n_tiles + 31) & ~31;
    return launch_pdl(k_shared_own_rows, (int64_t)t.own_chunks * pa.lh_count, kOwThreads, ow_bytes(tile_keys), pdl, s,
                      map(t.tmap_k), map(t.tmap_v), a, *t.reqs, pa, *t.groups, t.own_per_cta, tile_keys);
}

}  // namespace kvr
