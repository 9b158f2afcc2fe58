// kvr_key_weights_tc.cu -- attention weight per cached key on the tensor cores
// (bf16, head_dim 128).
//
// For every (request, layer, kv-head) and key row j < n = P_b + Lq_b:
//     w[j] (+)= sum over query rows r of exp2(c s_rj - lse_r),  s_rj = <rot(q_r), k_j>,
//     lse_r = log2 sum_j exp2(c s_rj),                          c = scale log2(e),
// a query row r being one of the G heads of one query token.
//
// The scores are computed the other way round, S^T = K Q^T: a 128-key tile is
// the M side of tcgen05.mma and the NQ query rows its N side.  A thread then
// owns a key (a TMEM lane): the sum over queries that makes a weight runs
// inside the thread, a decode step's few rows cost a narrow MMA instead of 128
// padded ones, and rows of the cache behind n stay in their own lanes.  Only
// the queries' denominators cross lanes, once per CTA.
//
// Every weight needs its rows' denominators over all keys before it can be
// summed.  So that K is read once, the scores stay in TMEM in between: of a
// CTA's 256 columns some 64 to 96 take the products, and the others hold the
// scores of tiles, one column a query row (48 tiles at up to 4 rows, 24 at 8, 10
// at 16, 5 at 32); the CTAs of a cluster split a unit's key tiles and exchange
// their rows' (max, sum) through distributed shared memory.  Tiles beyond what
// TMEM holds are processed first, for their statistics only, and loaded again at
// the end.
//
// Rotated queries are split into three bf16 terms (8 + 8 + 8 bits: all of the
// fp32 rotation's), so that the weights are fp32 results.  The terms stand side
// by side on the N side, and their products are added in registers: an MMA this
// narrow is bound by reading its 128-key operand from shared memory, once for
// the three.
//
// Two CTAs per SM (110 KB of shared memory, 256 TMEM columns each): one loads
// while the other is in its prologue or exchange.  Warps 0-3 rotate the
// queries and run the softmax passes; warp 4 issues the TMA loads (16 KB
// panels: 128 keys x 64 dims); warp 5 the MMAs.  All waits are bounded.
//
// Bound by the one read of K where it is long: 4 rows, 33,281 keys, 512 units:
// 721-745 us, 6.0-6.2 TB/s.  A short unit is latency: 7 rows, 2,657 keys, 112 units: 21
// us a call, 3.7 TB/s (setup and rotation 4 us, then two passes and an exchange
// that only the SM's other CTA overlaps).
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "kvr_tc_common.cuh"

namespace kvr {

namespace {

using namespace tc;

constexpr int kWtThreads = 192;
constexpr int kWtD = 128;
constexpr int kWtTile = 128;                 // keys per tile
constexpr int kWtPanel = kWtTile * 64 * 2;   // 16 KB: 128 keys x 64 dims
constexpr int kWtTmemCols = 256;
constexpr int kWtMaxCluster = 8;   // (16 CTAs, not portable: 1.31 ms against 1.03 on two 33k-token caches)
// a row that has seen no key yet: finite, so that the first score is far above
// it and sets the reference, and a masked -inf stays -inf
constexpr float kWtUnset = -1e30f;
constexpr float kWtHeadroom = 60.f;          // log2 units above the reference before it moves

// NC: query rows, padded to 4, 8, 16 or 32.
template <int NC>
struct WtCfg {
    static constexpr int kTermRows = NC < 8 ? 8 : NC;                // rows of a query term in the MMA operand
    static constexpr int NQ = (3 * kTermRows + 15) & ~15;            // columns of the S^T product: the three terms side by side
    static constexpr int kSlots = NC == 32 ? 5 : 6;                  // K panels in flight
    static constexpr int kStages = NC == 32 ? 1 : 2;                 // products in TMEM that wait for pass 1
    static constexpr int kKept = (kWtTmemCols - kStages * NQ) / NC;  // tiles whose scores stay in TMEM behind them
    static constexpr int kMaxCluster = NC == 32 ? 4 : kWtMaxCluster;
    static constexpr int kQPanel = NQ * 128;                         // the terms' rows x 64 dims
    static constexpr int kOffRing = 2 * kQPanel;
    static constexpr int kOffBar = kOffRing + kSlots * kWtPanel;
    // full[slots], empty[slots], s_full[stages], s_free[stages], q_full, peers, drain
    static constexpr int kNumBars = 2 * kSlots + 2 * kStages + 3;
    static constexpr int kOffMisc = kOffBar + 8 * kNumBars;          // TMEM address, abort flag
    static constexpr int kOffRef = (kOffMisc + 8 + 15) & ~15;        // [4][NC] reference per warp
    static constexpr int kOffStat = kOffRef + 4 * NC * 4;            // [4][NC] (reference, sum) per warp
    static constexpr int kOffFin = kOffStat + 4 * NC * 8;            // [NC] lse
    static constexpr int kOffPeer = kOffFin + NC * 4;                // [kMaxCluster][NC] (max, sum)
    static constexpr int kSmem = kOffPeer + kMaxCluster * NC * 8;
    static_assert(kSmem <= 113 * 1024, "two CTAs per SM");
};

// Order-preserving integer of a float (a warp's maximum by one integer reduction).
__device__ __forceinline__ int f_key(float x)
{
    const int i = __float_as_int(x);
    return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float key_f(int k) { return __int_as_float(k ^ ((k >> 31) & 0x7fffffff)); }

// Sums over the warp of NV values per lane; lane i gets value i % NV's (NV <= 32).
template <int NV>
__device__ __forceinline__ float warp_sums(float *v, int lane)
{
    int o = 16;
#pragma unroll
    for (int n = NV; n > 1; n >>= 1, o >>= 1) {
        // lanes with bit `o` take the upper half of the values
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float keep = up ? v[n / 2 + i] : v[i], give = up ? v[i] : v[n / 2 + i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    }
    float r = v[0];
#pragma unroll
    for (; o > 0; o >>= 1)
        r += __shfl_xor_sync(0xffffffffu, r, o);
    return r;
}
// The value that warp_sums<NV> leaves in `lane`.
template <int NV>
__device__ __forceinline__ int warp_sums_index(int lane)
{
    int idx = 0, o = 16;
#pragma unroll
    for (int n = NV; n > 1; n >>= 1, o >>= 1)
        idx += (lane & o) ? n / 2 : 0;
    return idx;
}

__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// (cos, sin) of pairs 8j .. 8j + 7 at position pos (interleaved: 4j .. 4j + 3 and
// 32 + 4j .. 32 + 4j + 3), as rope_cs, by 16-byte loads.
__device__ __forceinline__ void rope_cs8(const float2 *__restrict__ tab, int pos, int j, bool il, float2 *cs)
{
    const int p0 = il ? 4 * j : 8 * j, p1 = il ? 32 + 4 * j : 8 * j + 4;
    auto load = [&](int row, float4 *f) {
        const float2 *r = tab + row * (kWtD / 2);
        f[0] = __ldg(reinterpret_cast<const float4 *>(r + p0));
        f[1] = __ldg(reinterpret_cast<const float4 *>(r + p0) + 1);
        f[2] = __ldg(reinterpret_cast<const float4 *>(r + p1));
        f[3] = __ldg(reinterpret_cast<const float4 *>(r + p1) + 1);
    };
    float4 f[4];
    load(kRopeSplit + (pos & (kRopeSplit - 1)), f);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        cs[2 * e] = make_float2(f[e].x, f[e].y);
        cs[2 * e + 1] = make_float2(f[e].z, f[e].w);
    }
    if (pos >= kRopeSplit) {
        load(pos >> 12, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float hx = e & 1 ? f[e >> 1].z : f[e >> 1].x, hy = e & 1 ? f[e >> 1].w : f[e >> 1].y;
            cs[e] = make_float2(fmaf(hx, cs[e].x, -hy * cs[e].y), fmaf(hy, cs[e].x, hx * cs[e].y));
        }
    }
}

// Query rows r0 .. r0 + nr - 1 of a unit, rotated in fp32 and split into TERMS
// bf16 terms (what a term leaves goes to the next), written as K-major
// 128B-swizzled operands of ROWS rows (a multiple of 8): two 64-dim panels a
// term.  Rows past nr are zero.  128 threads; thread: RoPE pairs 8j .. 8j + 7,
// j = thread % 8, of a token's heads, four heads at a time (their angles are the
// same, and shared memory leaves next to no L1 that would keep a table row
// between them: a row at a time, a window's 128 rows took 17,000 cycles).
template <int TERMS, int ROWS>
__device__ __forceinline__ void prepare_queries(const WeightsArgs &a, const DevReq &rq, int l, int h, int G, int r0, int nr,
                                                uint32_t dst0, uint32_t term_bytes, uint32_t panel_bytes)
{
    const int j = threadIdx.x & 7, t_a = r0 / G, n_tok = (r0 + nr - 1) / G - t_a + 1;
    for (int it = threadIdx.x >> 3; it < n_tok; it += 16) {
        const int t = t_a + it;
        const __nv_bfloat16 *qp = static_cast<const __nv_bfloat16 *>(a.q) +
                                  (((int64_t)l * a.total_q + rq.q_off + t) * a.n_q_heads + h * G) * kWtD + 8 * j;
        const int row_t = t * G - r0;   // the row of head 0 (negative: in the block before)
        float2 cs[8];
        rope_cs8(a.rope, rq.prefix + t, j, a.interleaved, cs);
#pragma unroll 1
        for (int g0 = max(0, -row_t); g0 < G && row_t + g0 < nr; g0 += 4) {
            uint4 u[4][2];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const bool in = g0 + k < G && row_t + g0 + k < nr;
                const __nv_bfloat16 *p = qp + (in ? g0 + k : g0) * kWtD;
                u[k][0] = *reinterpret_cast<const uint4 *>(p);
                u[k][1] = *reinterpret_cast<const uint4 *>(p + 64);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int row = row_t + g0 + k;
                if (g0 + k >= G || row >= nr)
                    break;
                float v[16];   // elements 8j..8j+7 and 64+8j..64+8j+7
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t w4[4] = {u[k][x].x, u[k][x].y, u[k][x].z, u[k][x].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[8 * x + 2 * e] = __uint_as_float(w4[e] << 16);
                        v[8 * x + 2 * e + 1] = __uint_as_float(w4[e] & 0xffff0000u);
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float x0 = a.interleaved ? v[2 * e] : v[e], x1 = a.interleaved ? v[2 * e + 1] : v[8 + e];
                    const float y0 = fmaf(x0, cs[e].x, -x1 * cs[e].y), y1 = fmaf(x0, cs[e].y, x1 * cs[e].x);
                    if (a.interleaved) {
                        v[2 * e] = y0;
                        v[2 * e + 1] = y1;
                    } else {
                        v[e] = y0;
                        v[8 + e] = y1;
                    }
                }
                const uint32_t dst = dst0 + (uint32_t)(row * 128 + ((j ^ (row & 7)) << 4));
#pragma unroll
                for (int term = 0; term < TERMS; ++term)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        uint32_t w4[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float &x0 = v[8 * x + 2 * e], &x1 = v[8 * x + 2 * e + 1];
                            const __nv_bfloat162 b = __floats2bfloat162_rn(x0, x1);
                            w4[e] = *reinterpret_cast<const uint32_t *>(&b);
                            x0 -= __low2float(b);    // exact: what the term leaves
                            x1 -= __high2float(b);
                        }
                        st_shared_v4(dst + (uint32_t)term * term_bytes + (uint32_t)x * panel_bytes, w4[0], w4[1], w4[2], w4[3]);
                    }
            }
        }
    }
    for (int row = nr + (int)(threadIdx.x >> 3); row < ROWS; row += 16)
#pragma unroll
        for (int term = 0; term < TERMS; ++term)
#pragma unroll
            for (int x = 0; x < 2; ++x)
                st_shared_v4(dst0 + (uint32_t)(row * 128 + (j << 4)) + (uint32_t)term * term_bytes + (uint32_t)x * panel_bytes, 0u,
                             0u, 0u, 0u);
}

// Bounded wait that sees what other CTAs of the cluster released before arriving.
__device__ __forceinline__ bool wait_peers(uint32_t bar, uint32_t parity, volatile int *abort_flag)
{
    const uint64_t t0 = globaltimer();
    while (true) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok)
            return true;
        if (*abort_flag || globaltimer() - t0 > kWaitNs)
            return false;
    }
}

}  // namespace

template <int NC>
__global__ void __launch_bounds__(kWtThreads, 2)
    k_key_weights_tc(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ WeightsArgs a,
                     const __grid_constant__ ReqTable rt, const int n_cluster)
{
    using C = WtCfg<NC>;
    constexpr int NQ = C::NQ;
    constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(NQ >> 3) << 17) |
                                ((uint32_t)(kWtTile >> 4) << 24);
    extern __shared__ __align__(1024) uint8_t wt_smem[];
    const uint32_t sbase = smem_u32(wt_smem);
    auto bar = [&](int i) { return sbase + C::kOffBar + 8u * (uint32_t)i; };
    constexpr int bFull = 0, bEmpty = C::kSlots, bSFull = 2 * C::kSlots, bSFree = bSFull + C::kStages,
                  bQFull = bSFree + C::kStages, bPeers = bQFull + 1, bDrain = bQFull + 2;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(wt_smem + C::kOffMisc + 4);
    float *s_ref = reinterpret_cast<float *>(wt_smem + C::kOffRef);
    float2 *s_stat = reinterpret_cast<float2 *>(wt_smem + C::kOffStat);
    float *s_fin = reinterpret_cast<float *>(wt_smem + C::kOffFin);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int units = a.n_layers * a.n_kv_heads;
    const int rank = (int)(blockIdx.x % (unsigned)n_cluster), unit_i = (int)(blockIdx.x / (unsigned)n_cluster);

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kNumBars; ++i) {
            const bool wg = (i >= bSFree && i < bSFree + C::kStages) || i == bQFull;
            mbar_init(bar(i), wg ? 128u : i == bPeers ? (uint32_t)(n_cluster * NC) : 1u);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 5)
        tmem_alloc(sbase + C::kOffMisc, kWtTmemCols);
    if (warp == 4 && lane == 0)
        prefetch_tmap(&tmk);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (n_cluster > 1)
        cluster_sync();   // the peers' barriers are initialised before any remote arrive
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(wt_smem + C::kOffMisc);
    pdl_wait_prerequisites();

    const DevReq *reqs = a.reqs ? a.reqs : rt.reqs;
    const DevReq rq = reqs[a.req0 + unit_i / units];
    const int lh = unit_i % units;
    const int G = a.n_q_heads / a.n_kv_heads;
    const int m_rows = rq.q_len * G, n = rq.prefix + rq.q_len;
    const int nt = (n + kWtTile - 1) / kWtTile;
    const int t_lo = (int)((int64_t)rank * nt / n_cluster), t_hi = (int)((int64_t)(rank + 1) * nt / n_cluster);
    const int T = t_hi - t_lo;                               // this CTA's key tiles
    const int n_redo = max(0, T - C::kKept);                 // loaded a second time
    const int64_t blk = rq.cache_row0 + (int64_t)lh * rq.cap;
    // job i: tiles T-1 .. 0 for the statistics, then kKept .. T-1 again; its
    // product goes to stage i % kStages
    auto job_tile = [&](int i) { return i < T ? T - 1 - i : C::kKept + (i - T); };
    const int n_jobs = m_rows > 0 ? T + n_redo : 0;

    if (warp < 4) {
        const int l = lh / a.n_kv_heads, h = lh - l * a.n_kv_heads;
        const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
        const float sc = a.scale_log2;
        float *wp = a.weights + blk;
        int job = 0;
        bool ok = true;
        if (m_rows == 0 && !a.accumulate)   // a sum over no queries
            for (int j = t_lo * kWtTile + (int)threadIdx.x; j < min(n, t_hi * kWtTile); j += 128)
                wp[j] = 0.f;
        if (m_rows > 0) {   // the same for the whole cluster; at most NC rows
            // ---- the queries: rotated, split in three bf16 terms ----
            prepare_queries<3, C::kTermRows>(a, rq, l, h, G, 0, m_rows, sbase, (uint32_t)(C::kTermRows * 128), (uint32_t)C::kQPanel);
            fence_proxy_async_smem();
            mbar_arrive(bar(bQFull));

            // NC columns at a TMEM address; keys that a row does not see are -inf.
            // lim: the first column that sees this key.
            auto load = [&](uint32_t at, float *s) {
                if constexpr (NC == 4)
                    tmem_ld4(at, s);
                else if constexpr (NC == 8)
                    tmem_ld8(at, s);
                else if constexpr (NC == 16)
                    tmem_ld16(at, s);
                else
                    tmem_ld32(at, s);
            };
            auto keep = [&](uint32_t at, const float *s) {
                if constexpr (NC == 4)
                    tmem_st4(at, s);
                else if constexpr (NC == 8)
                    tmem_st8(at, s);
                else if constexpr (NC == 16)
                    tmem_st16(at, reinterpret_cast<const uint32_t *>(s));
                else
                    tmem_st32(at, s);
            };
            // a product: the sum of the three terms'
            auto load_job = [&](int jb, float *s) {
                const uint32_t at = lane_base + (uint32_t)((jb % C::kStages) * NQ);
                float mid[NC], low[NC];
                load(at, s);
                load(at + C::kTermRows, mid);
                load(at + 2 * C::kTermRows, low);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    s[c] += mid[c] + low[c];
            };
            auto wait_job = [&](int jb) -> bool {
                if (!mbar_wait_warp(bar(bSFull + jb % C::kStages), (uint32_t)(jb / C::kStages) & 1, abort_flag))
                    return false;
                tc_fence_after();
                return true;
            };
            auto free_job = [&](int jb) {
                tc_fence_before();
                mbar_arrive(bar(bSFree + jb % C::kStages));
            };
            auto mask = [&](int lim, float *s) {
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    s[c] = c >= lim ? s[c] : -INFINITY;
            };
            // scores kept of tile t
            auto kept_at = [&](int t) { return lane_base + (uint32_t)(C::kStages * NQ + t * NC); };

            // ---- pass 1: each row's reference and sum over this warp's keys ----
            float ls[NC];
#pragma unroll
            for (int c = 0; c < NC; ++c)
                ls[c] = 0.f;
            float *ref = s_ref + warp * NC;
            if (lane < NC)
                ref[lane] = kWtUnset;
            __syncwarp();
            for (int i = 0; i < T; ++i, ++job) {
                const int t = T - 1 - i;
                if (!wait_job(job)) {
                    ok = false;
                    break;
                }
                const int j0 = (t_lo + t) * kWtTile, j = j0 + (int)threadIdx.x;
                const bool edge = j0 + kWtTile > rq.prefix + 1;   // some key is not seen by every row
                float s[NC];
                load_job(job, s);
                if (t < C::kKept)   // uniform
                    keep(kept_at(t), s);
                free_job(job);
                if (edge)
                    mask(j >= n ? NC : (j - rq.prefix) * G, s);
                float mx = -INFINITY;
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    s[c] *= sc;
                    mx = fmaxf(mx, s[c] - ref[c]);
                }
                if (__any_sync(0xffffffffu, mx > kWtHeadroom)) {
                    // a first key, or one far above the reference: the rows'
                    // references move up to this tile's maxima
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        const float old = ref[c];
                        const float m = key_f(__reduce_max_sync(0xffffffffu, f_key(s[c])));
                        if (m > old) {   // the same in all lanes
                            ls[c] = old == kWtUnset ? 0.f : ls[c] * ex2(old - m);
                            __syncwarp();
                            if (lane == 0)
                                ref[c] = m;
                            __syncwarp();
                        }
                    }
                }
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    ls[c] += ex2(s[c] - ref[c]);
            }
            // (a thread whose wait ran out goes on to the barriers below with the others)
            if (!ok)
                give_up(a.err, abort_flag);
            tmem_wait_st();
            {
                const float r = warp_sums<NC>(ls, lane);
                const int c = warp_sums_index<NC>(lane);
                s_stat[warp * NC + c] = make_float2(ref[c], r);
            }
            softmax_sync();
            // ---- the CTA's (max, sum) of row c to every CTA of the cluster ----
            const uint32_t peer = sbase + C::kOffPeer;
            if (threadIdx.x < NC) {
                const int c = threadIdx.x;
                float M = kWtUnset, L = 0.f;
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    M = fmaxf(M, s_stat[x * NC + c].x);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float2 v = s_stat[x * NC + c];
                    L += v.y != 0.f ? v.y * ex2(v.x - M) : 0.f;
                }
                for (int x = 0; x < n_cluster; ++x) {
                    const uint32_t dst = mapa_rank(peer + (uint32_t)((rank * NC + c) * 8), (uint32_t)x);
                    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(dst), "f"(M), "f"(L) : "memory");
                    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                                     mapa_rank(bar(bPeers), (uint32_t)x))
                                 : "memory");
                }
                if (wait_peers(bar(bPeers), 0, abort_flag)) {
                    float Mt = kWtUnset, Lt = 0.f;
                    const float2 *pv = reinterpret_cast<const float2 *>(wt_smem + C::kOffPeer) + c;
                    for (int x = 0; x < n_cluster; ++x)
                        Mt = fmaxf(Mt, pv[x * NC].x);
                    for (int x = 0; x < n_cluster; ++x) {   // in rank order: one rounding order
                        const float2 v = pv[x * NC];
                        Lt += v.y != 0.f ? v.y * ex2(v.x - Mt) : 0.f;
                    }
                    s_fin[c] = Mt + log2f(Lt);
                    if (c < m_rows && rank == 0 && !(Lt > 0.f && Lt < INFINITY))
                        atomicCAS(a.err, kDevOk, kDevBadInput);
                } else {
                    give_up(a.err, abort_flag);
                }
            }
            softmax_sync();
            // (one answer for the warp's tcgen05 loads: a peer or another role may set the
            // flag between two lanes' reads)
            if (__any_sync(0xffffffffu, *abort_flag != 0))
                ok = false;
            // ---- pass 2: the weights of this thread's keys ----
            // (the weights to add to are read eight tiles ahead)
            float old[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            for (int t = 0; t < T && ok; ++t) {
                const int j0 = (t_lo + t) * kWtTile, j = j0 + (int)threadIdx.x;
                if (a.accumulate && (t & 7) == 0) {
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        old[x] = t + x < T && j + x * kWtTile < n ? wp[j + x * kWtTile] : 0.f;
                }
                const float w = old[0];
#pragma unroll
                for (int x = 0; x < 7; ++x)
                    old[x] = old[x + 1];
                const bool redo = t >= C::kKept;
                if (redo && !wait_job(job)) {
                    ok = false;
                    break;
                }
                float s[NC], p4[4] = {0.f, 0.f, 0.f, 0.f};
                if (redo) {
                    load_job(job, s);
                    free_job(job);
                    ++job;
                } else {
                    load(kept_at(t), s);
                    tmem_wait_ld();
                }
                if (j0 + kWtTile > rq.prefix + 1)
                    mask(j >= n ? NC : (j - rq.prefix) * G, s);
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    p4[c & 3] += c < m_rows ? ex2(fmaf(s[c], sc, -s_fin[c])) : 0.f;
                if (j < n)
                    wp[j] = w + ((p4[0] + p4[1]) + (p4[2] + p4[3]));
            }
        }
        if (!ok)
            give_up(a.err, abort_flag);
    } else if (warp == 4) {
        if (lane == 0) {
            bool ok = true;
            int k = 0;   // panels issued
            for (int i = 0; i < n_jobs && ok; ++i) {
                const int row = (int)(blk + (int64_t)(t_lo + job_tile(i)) * kWtTile);
                for (int p = 0; p < 2; ++p, ++k) {
                    const int s = k % C::kSlots;
                    if (k >= C::kSlots && !mbar_wait(bar(bEmpty + s), (uint32_t)(k / C::kSlots - 1) & 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    mbar_expect_tx(bar(bFull + s), kWtPanel);
                    tma_load_2d(sbase + (uint32_t)(C::kOffRing + s * kWtPanel), &tmk, 64 * p, row, bar(bFull + s));
                }
            }
            if (!ok)
                give_up(a.err, abort_flag);
            // every issued copy lands before the CTA leaves
            for (int x = k > C::kSlots ? k - C::kSlots : 0; x < k; ++x)
                mbar_drain(bar(bFull + x % C::kSlots), (uint32_t)(x / C::kSlots) & 1);
        }
    } else {
        const uint32_t lead = elect_one();
        const uint64_t d0 = sdesc(sbase, 16, 1024);
        const uint32_t lo = (uint32_t)d0, hi = (uint32_t)(d0 >> 32);
        bool ok = n_jobs == 0 || mbar_wait_warp(bar(bQFull), 0, abort_flag);
        int k = 0;
        for (int i = 0; i < n_jobs && ok; ++i) {
            const int stage = i % C::kStages;
            if (i >= C::kStages && !mbar_wait_warp(bar(bSFree + stage), (uint32_t)(i / C::kStages - 1) & 1, abort_flag)) {
                ok = false;
                break;
            }
            for (int p = 0; p < 2; ++p, ++k) {
                const int s = k % C::kSlots;
                if (!mbar_wait_warp(bar(bFull + s), (uint32_t)(k / C::kSlots) & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t ka = lo + ((uint32_t)(C::kOffRing + s * kWtPanel) >> 4);
                const uint32_t qb = lo + ((uint32_t)(p * C::kQPanel) >> 4);
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    mma_ss(lead, tmem + (uint32_t)(stage * NQ), desc_with_lo(ka + 2 * x, hi), desc_with_lo(qb + 2 * x, hi), kIdesc,
                           p > 0 || x > 0);
                umma_commit(lead, bar(bEmpty + s));
            }
            if (ok)
                umma_commit(lead, bar(bSFull + stage));
        }
        if (!ok)
            give_up(a.err, abort_flag);
        // all issued MMAs complete before TMEM is released
        umma_commit(lead, bar(bDrain));
        mbar_drain(bar(bDrain), 0);
    }
    tc_fence_before();
    __syncthreads();
    if (n_cluster > 1)
        cluster_sync();   // no CTA leaves while a peer may still write to its shared memory
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc(tmem, kWtTmemCols);
    }
}

// ---------------------------------------------------------------------------
// windows: more than 32 query rows
// ---------------------------------------------------------------------------
// At many rows the scores of a unit do not fit TMEM, and the products, not the
// read of K, bound the kernel.  So K is streamed twice (the second time mostly
// from L2) and each pass takes the orientation in which its sum stays inside a
// thread: S = Q K^T for the rows' denominators (a thread owns a query row),
// S^T = K Q^T for the weights (a thread owns a key); the two operands' shared
// memory is the same.  Two bf16 query terms: the weight of a key sums over all
// the rows, which averages the 2^-17 that they leave.  Blocks of 128 rows; a
// unit's tiles are split over a cluster only when there are too few units to
// fill the SMs.  128 rows, 969 to 1,248 keys, 4,608 units: 483 us in single
// calls, 533-548 in runs long enough for the power cap; the 2 x 2
// products are 340 us at the tensor rate, and a fifth of a CTA's time is setup,
// rotation and exit, which only the SM's other CTA overlaps.  (32 rows cost it
// 434 us on 16 requests of 1,300 keys, the kernel above 375; that one, with 128
// rows' scores in TMEM, would keep one tile.)
namespace {
constexpr int kWwSlots = 3;
constexpr int kWwMaxCluster = 8;
constexpr int kWwQTerm = 128 * kWtD * 2;
constexpr int kWwOffRing = 2 * kWwQTerm;
constexpr int kWwOffBar = kWwOffRing + kWwSlots * kWtPanel;
constexpr int kWwNumBars = 2 * kWwSlots + 4 + 5;   // full, empty, s_full[2], s_free[2], q_full, q_empty, peers[2], drain
constexpr int kWwOffMisc = kWwOffBar + 8 * kWwNumBars;
constexpr int kWwOffFin = (kWwOffMisc + 12 + 15) & ~15;         // [128] -lse
constexpr int kWwSmem = kWwOffFin + 128 * 4;
constexpr int kWwOffPeer = kWwSmem;                            // [2][kWwMaxCluster][128] (max, sum), clusters only
constexpr int kWwSmemCluster = kWwOffPeer + 2 * kWwMaxCluster * 128 * 8;
static_assert(kWwSmem <= 113 * 1024, "two CTAs per SM");
}  // namespace

__global__ void __launch_bounds__(kWtThreads, 2)
    k_key_weights_window(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ WeightsArgs a,
                         const __grid_constant__ ReqTable rt, const int n_cluster)
{
    constexpr uint32_t kIdescBase = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kWtTile >> 4) << 24);
    extern __shared__ __align__(1024) uint8_t wt_smem[];
    const uint32_t sbase = smem_u32(wt_smem);
    auto bar = [&](int i) { return sbase + kWwOffBar + 8u * (uint32_t)i; };
    constexpr int bFull = 0, bEmpty = kWwSlots, bSFull = 2 * kWwSlots, bSFree = bSFull + 2, bQFull = bSFree + 2,
                  bQEmpty = bQFull + 1, bPeers = bQFull + 2, bDrain = bPeers + 2;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(wt_smem + kWwOffMisc + 4), *abort_seen = abort_flag + 1;
    float *s_fin = reinterpret_cast<float *>(wt_smem + kWwOffFin);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int units = a.n_layers * a.n_kv_heads;
    const int rank = (int)(blockIdx.x % (unsigned)n_cluster), unit_i = (int)(blockIdx.x / (unsigned)n_cluster);

    if (threadIdx.x == 0) {
        for (int i = 0; i < kWwNumBars; ++i)
            mbar_init(bar(i), (i >= bSFree && i < bSFree + 2) || i == bQFull  ? 128u
                              : i >= bPeers && i < bPeers + 2 ? (uint32_t)(n_cluster * 128)
                                                              : 1u);
        *abort_flag = *abort_seen = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 5)
        tmem_alloc(sbase + kWwOffMisc, kWtTmemCols);
    if (warp == 4 && lane == 0)
        prefetch_tmap(&tmk);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (n_cluster > 1)
        cluster_sync();   // the peers' barriers are initialised before any remote arrive
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(wt_smem + kWwOffMisc);
    pdl_wait_prerequisites();

    const DevReq *reqs = a.reqs ? a.reqs : rt.reqs;
    const DevReq rq = reqs[a.req0 + unit_i / units];
    const int lh = unit_i % units;
    const int G = a.n_q_heads / a.n_kv_heads;
    const int m_rows = rq.q_len * G, n = rq.prefix + rq.q_len;
    const int n_rb = (m_rows + 127) / 128;
    const int nt = (n + kWtTile - 1) / kWtTile;
    const int t_lo = (int)((int64_t)rank * nt / n_cluster), t_hi = (int)((int64_t)(rank + 1) * nt / n_cluster);
    const int T = t_hi - t_lo;
    const int64_t blk = rq.cache_row0 + (int64_t)lh * rq.cap;
    // job i of a row block: tiles 0 .. T-1, then T-1 .. 0; scores in TMEM half i & 1
    auto job_tile = [&](int i) { return i < T ? i : 2 * T - 1 - i; };

    if (warp < 4) {
        const int l = lh / a.n_kv_heads, h = lh - l * a.n_kv_heads;
        const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
        const float sc = a.scale_log2;
        float *wp = a.weights + blk;
        int job = 0;   // over all row blocks (2 T is even: the halves alternate on)
        bool ok = true;
        if (m_rows == 0 && !a.accumulate)
            for (int j = t_lo * kWtTile + (int)threadIdx.x; j < min(n, t_hi * kWtTile); j += 128)
                wp[j] = 0.f;
        // (a thread whose wait ran out still passes every barrier of the 128, until
        // all of them leave together)
        for (int rb = 0; rb < n_rb; ++rb) {
            const int r0 = rb * 128, nr = min(128, m_rows - r0);
            ok = ok && (rb == 0 || mbar_wait_warp(bar(bQEmpty), (uint32_t)(rb - 1) & 1, abort_flag));
            prepare_queries<2, 128>(a, rq, l, h, G, r0, nr, sbase, (uint32_t)kWwQTerm, (uint32_t)(kWwQTerm / 2));
            fence_proxy_async_smem();
            mbar_arrive(bar(bQFull));

            // ---- pass 1: this thread's query row over the CTA's keys ----
            const int r = threadIdx.x;
            const int see = rq.prefix + (r0 + min(r, nr - 1)) / G + 1;   // keys the row sees
            float m = kWtUnset, lsum = 0.f;
            for (int i = 0; i < T && ok; ++i, ++job) {
                const int half = job & 1;
                if (!mbar_wait_warp(bar(bSFull + half), (uint32_t)(job >> 1) & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (warp * 32 < nr) {
                    const int lim = see - (t_lo + i) * kWtTile;
                    const uint32_t at = lane_base + (uint32_t)(half * 128);
                    auto block = [&](int q, float *s) {
                        if (lim < kWtTile) {
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                s[c] = q * 32 + c < lim ? s[c] : -INFINITY;
                        }
                        float m4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                        for (int c = 4; c < 28; c += 8)
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                m4[x] = max3(m4[x], s[c + 2 * x], s[c + 2 * x + 1]);
                        const float mx = max3(max3(m4[0], m4[1], s[28]), max3(m4[2], m4[3], s[29]), fmaxf(s[30], s[31])) * sc;
                        if (mx > m + 8.f) {   // (the reference need not be the maximum)
                            lsum = lsum == 0.f ? 0.f : lsum * ex2(m - mx);
                            m = mx;
                        }
                        const uint64_t sc2 = pk2(sc, sc), nm2 = pk2(-m, -m);
                        uint64_t acc[2] = {pk2(0.f, 0.f), pk2(0.f, 0.f)};
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            float x0, x1;
                            unpk2(fma2(pk2(s[2 * c], s[2 * c + 1]), sc2, nm2), x0, x1);
                            acc[c & 1] = add2(acc[c & 1], pk2(ex2(x0), ex2(x1)));
                        }
                        float a0, a1, b0, b1;
                        unpk2(acc[0], a0, a1);
                        unpk2(acc[1], b0, b1);
                        lsum += (a0 + a1) + (b0 + b1);
                    };
                    // the next 32 columns are on their way while these are summed
                    float sa[32], sb[32];
                    tmem_ld32(at, sa);
                    tmem_wait_ld();
                    tmem_ld32(at + 32, sb);
                    block(0, sa);
                    tmem_wait_ld();
                    tmem_ld32(at + 64, sa);
                    block(1, sb);
                    tmem_wait_ld();
                    tmem_ld32(at + 96, sb);
                    block(2, sa);
                    tmem_wait_ld();
                    block(3, sb);
                }
                tc_fence_before();
                mbar_arrive(bar(bSFree + half));
            }
            if (!ok)
                give_up(a.err, abort_flag);
            float M = m, L = lsum;
            if (n_cluster > 1) {
                // Row blocks take two barriers and two sets of places by turns.  A phase that
                // is complete here says that every thread has arrived here, not at the other
                // CTAs: with one barrier, this CTA's arrivals for block rb + 1 could count at a
                // CTA that a slower thread's arrival for rb has yet to reach.  With two, the
                // arrivals for rb + 2 come after a wait for rb + 1, which every thread joins
                // only after its arrivals for rb.
                const int turn = rb & 1;
                const uint32_t peer = sbase + kWwOffPeer + (uint32_t)(turn * kWwMaxCluster * 128 * 8);
                for (int x = 0; x < n_cluster; ++x) {
                    const uint32_t dst = mapa_rank(peer + (uint32_t)((rank * 128 + r) * 8), (uint32_t)x);
                    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(dst), "f"(m), "f"(lsum) : "memory");
                    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                                     mapa_rank(bar(bPeers + turn), (uint32_t)x))
                                 : "memory");
                }
                if (wait_peers(bar(bPeers + turn), (uint32_t)(rb >> 1) & 1, abort_flag)) {
                    const float2 *pv = reinterpret_cast<const float2 *>(wt_smem + kWwOffPeer) + turn * kWwMaxCluster * 128 + r;
                    M = kWtUnset;
                    L = 0.f;
                    for (int x = 0; x < n_cluster; ++x)
                        M = fmaxf(M, pv[x * 128].x);
                    for (int x = 0; x < n_cluster; ++x) {   // in rank order: one rounding order
                        const float2 v = pv[x * 128];
                        L += v.y != 0.f ? v.y * ex2(v.x - M) : 0.f;
                    }
                } else {
                    give_up(a.err, abort_flag);
                }
            }
            softmax_sync();   // (the row block before has read its denominators)
            s_fin[r] = r < nr ? -(M + log2f(L)) : 0.f;   // (rows that pad the block: any finite value)
            if (r < nr && rank == 0 && !(L > 0.f && L < INFINITY))
                atomicCAS(a.err, kDevOk, kDevBadInput);
            if (threadIdx.x == 0)
                *abort_seen = *abort_flag;
            softmax_sync();
            if (*abort_seen) {   // the same for all 128 threads
                ok = false;
                break;
            }
            // ---- pass 2: the weights of this thread's keys ----
            const bool add = rb > 0 || a.accumulate;
            const int nb = (nr + 31) >> 5;   // 32-row blocks of queries
            for (int i = 0; i < T && ok; ++i, ++job) {
                const int half = job & 1;
                const int j0 = (t_lo + T - 1 - i) * kWtTile, j = j0 + (int)threadIdx.x;
                const float w = add && j < n ? wp[j] : 0.f;
                if (!mbar_wait_warp(bar(bSFull + half), (uint32_t)(job >> 1) & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const bool edge = j0 + kWtTile > rq.prefix + 1;
                const int lim = !edge ? 0 : j >= n ? 128 : (j - rq.prefix) * G - r0;   // the first row that sees the key
                uint64_t acc[2] = {pk2(0.f, 0.f), pk2(0.f, 0.f)};
                const uint64_t sc2 = pk2(sc, sc);
                const uint32_t at = lane_base + (uint32_t)(half * 128);
                auto block = [&](int q, float *s) {
                    const int hi = nr - q * 32;
                    if (edge || hi < 32) {
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            s[c] = q * 32 + c >= lim && c < hi ? s[c] : -INFINITY;
                    }
                    const float4 *fin = reinterpret_cast<const float4 *>(s_fin + q * 32);   // -lse
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const float4 f = fin[c];
                        float x0, x1, x2, x3;
                        unpk2(fma2(pk2(s[4 * c], s[4 * c + 1]), sc2, pk2(f.x, f.y)), x0, x1);
                        unpk2(fma2(pk2(s[4 * c + 2], s[4 * c + 3]), sc2, pk2(f.z, f.w)), x2, x3);
                        acc[0] = add2(acc[0], pk2(ex2(x0), ex2(x1)));
                        acc[1] = add2(acc[1], pk2(ex2(x2), ex2(x3)));
                    }
                };
                float sa[32], sb[32];
                tmem_ld32(at, sa);
                tmem_wait_ld();
                if (nb > 1)   // the next 32 rows are on their way while these are summed
                    tmem_ld32(at + 32, sb);
                block(0, sa);
                tmem_wait_ld();
                if (nb > 1) {
                    if (nb > 2)
                        tmem_ld32(at + 64, sa);
                    block(1, sb);
                    tmem_wait_ld();
                    if (nb > 2) {
                        if (nb > 3)
                            tmem_ld32(at + 96, sb);
                        block(2, sa);
                        tmem_wait_ld();
                        if (nb > 3)
                            block(3, sb);
                    }
                }
                float a0, a1, b0, b1;
                unpk2(acc[0], a0, a1);
                unpk2(acc[1], b0, b1);
                const float sum = (a0 + a1) + (b0 + b1);
                tc_fence_before();
                mbar_arrive(bar(bSFree + half));
                if (j < n)
                    wp[j] = w + sum;
            }
        }
        if (!ok)
            give_up(a.err, abort_flag);
    } else if (warp == 4) {
        if (lane == 0) {
            bool ok = true;
            int k = 0;   // panels issued
            for (int rb = 0; rb < n_rb && ok; ++rb)
                for (int i = 0; i < 2 * T && ok; ++i) {
                    const int row = (int)(blk + (int64_t)(t_lo + job_tile(i)) * kWtTile);
                    for (int p = 0; p < 2; ++p, ++k) {
                        const int s = k % kWwSlots;
                        if (k >= kWwSlots && !mbar_wait(bar(bEmpty + s), (uint32_t)(k / kWwSlots - 1) & 1, abort_flag)) {
                            ok = false;
                            break;
                        }
                        mbar_expect_tx(bar(bFull + s), kWtPanel);
                        tma_load_2d(sbase + (uint32_t)(kWwOffRing + s * kWtPanel), &tmk, 64 * p, row, bar(bFull + s));
                    }
                }
            if (!ok)
                give_up(a.err, abort_flag);
            for (int x = k > kWwSlots ? k - kWwSlots : 0; x < k; ++x)
                mbar_drain(bar(bFull + x % kWwSlots), (uint32_t)(x / kWwSlots) & 1);
        }
    } else {
        const uint32_t lead = elect_one();
        const uint64_t d0 = sdesc(sbase, 16, 1024);
        const uint32_t lo = (uint32_t)d0, hi = (uint32_t)(d0 >> 32);
        bool ok = true;
        int k = 0, job = 0;
        for (int rb = 0; rb < n_rb && ok; ++rb) {
            if (!mbar_wait_warp(bar(bQFull), (uint32_t)rb & 1, abort_flag)) {
                ok = false;
                break;
            }
            const int nr = min(128, m_rows - rb * 128);
            const uint32_t idesc_t = kIdescBase | ((uint32_t)(((nr + 31) & ~31) >> 3) << 17);   // S^T: N = rows
            const uint32_t idesc_s = kIdescBase | ((uint32_t)(kWtTile >> 3) << 17);             // S: N = keys
            for (int i = 0; i < 2 * T && ok; ++i, ++job) {
                const int half = job & 1;
                if (job >= 2 && !mbar_wait_warp(bar(bSFree + half), (uint32_t)((job >> 1) - 1) & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                const bool second = i >= T;
                for (int p = 0; p < 2; ++p, ++k) {
                    const int s = k % kWwSlots;
                    if (!mbar_wait_warp(bar(bFull + s), (uint32_t)(k / kWwSlots) & 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t ka = lo + ((uint32_t)(kWwOffRing + s * kWtPanel) >> 4);
#pragma unroll
                    for (int term = 0; term < 2; ++term) {
                        const uint32_t qb = lo + ((uint32_t)(term * kWwQTerm + p * (kWwQTerm / 2)) >> 4);
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            mma_ss(lead, tmem + (uint32_t)(half * 128), desc_with_lo((second ? ka : qb) + 2 * x, hi),
                                   desc_with_lo((second ? qb : ka) + 2 * x, hi), second ? idesc_t : idesc_s,
                                   p > 0 || term > 0 || x > 0);
                    }
                    umma_commit(lead, bar(bEmpty + s));
                }
                if (ok)
                    umma_commit(lead, bar(bSFull + half));
            }
            umma_commit(lead, bar(bQEmpty));
        }
        if (!ok)
            give_up(a.err, abort_flag);
        umma_commit(lead, bar(bDrain));
        mbar_drain(bar(bDrain), 0);
    }
    tc_fence_before();
    __syncthreads();
    if (n_cluster > 1)
        cluster_sync();   // no CTA leaves while a peer may still write to its shared memory
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc(tmem, kWtTmemCols);
    }
}

template <int NC>
static cudaError_t launch_nq(const WeightsArgs &a, const ReqTable &rt, const CUtensorMap &tmk, int n_sms, cudaStream_t s)
{
    using C = WtCfg<NC>;
    static std::atomic<bool> attr_set[64] = {};   // per device (host threads may race: same value)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev >= 64 || !attr_set[dev].load(std::memory_order_acquire)) {
        if ((e = cudaFuncSetAttribute(k_key_weights_tc<NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem)) !=
                cudaSuccess ||
            (e = cudaFuncSetAttribute(k_key_weights_tc<NC>, cudaFuncAttributePreferredSharedMemoryCarveout, 100)) != cudaSuccess)
            return e;
        if (dev < 64)
            attr_set[dev].store(true, std::memory_order_release);
    }
    const int64_t units = (int64_t)a.n_reqs * a.n_layers * a.n_kv_heads;
    const int tiles = (a.max_rows + kWtTile - 1) / kWtTile;
    // A cluster's CTAs together keep more scores in TMEM, but each pays its
    // prologue and exchange: the cluster grows while the longest request's scores
    // do not fit and a CTA keeps ten tiles (288 units: 16 rows, 11 tiles: 25 us
    // with one CTA, 31 with two; 47 tiles: 116, 108, 100 and 128 with 1, 2, 4 and
    // 8; 258 tiles: 669, 654, 616 and 590.  32 rows: 4 CTAs at most, 258 tiles:
    // 651 with 4, 692 with 8).  And it grows while SMs would be idle and a CTA
    // keeps four tiles (112 units of 21 tiles: 28 us with 2, 34 with 4).
    int c = 1;
    while (c < C::kMaxCluster &&
           ((tiles > c * C::kKept && tiles >= 20 * c) || (units * c <= n_sms && tiles >= 8 * c)))
        c *= 2;
    return launch_cluster(k_key_weights_tc<NC>, units * c, kWtThreads, C::kSmem, c, s, tmk, a, rt, c);
}

static cudaError_t launch_window(const WeightsArgs &a, const ReqTable &rt, const CUtensorMap &tmk, int n_sms, cudaStream_t s)
{
    static std::atomic<bool> attr_set[64] = {};   // per device (host threads may race: same value)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev >= 64 || !attr_set[dev].load(std::memory_order_acquire)) {
        if ((e = cudaFuncSetAttribute(k_key_weights_window, cudaFuncAttributeMaxDynamicSharedMemorySize, kWwSmemCluster)) !=
                cudaSuccess ||
            (e = cudaFuncSetAttribute(k_key_weights_window, cudaFuncAttributePreferredSharedMemoryCarveout, 100)) != cudaSuccess)
            return e;
        if (dev < 64)
            attr_set[dev].store(true, std::memory_order_release);
    }
    const int64_t units = (int64_t)a.n_reqs * a.n_layers * a.n_kv_heads;
    const int tiles = (a.max_rows + kWtTile - 1) / kWtTile;
    int c = 1;   // split a unit's tiles while the grid leaves SMs idle (one CTA per SM then)
    while (c < kWwMaxCluster && units * c * 2 <= n_sms && tiles >= 4 * c)
        c *= 2;
    return launch_cluster(k_key_weights_window, units * c, kWtThreads, c > 1 ? kWwSmemCluster : kWwSmem, c, s, tmk, a, rt, c);
}

static_assert(kWeightsFewRows == 32, "the most rows of k_key_weights_tc");
cudaError_t launch_weights_tc(const WeightsArgs &a, const ReqTable &rt, const void *tmap_k, int n_sms, cudaStream_t s)
{
    const CUtensorMap &m = *static_cast<const CUtensorMap *>(tmap_k);
    const int64_t rows = (int64_t)a.max_q_len * (a.n_q_heads / a.n_kv_heads);
    if (rows <= 4)
        return launch_nq<4>(a, rt, m, n_sms, s);
    if (rows <= 8)
        return launch_nq<8>(a, rt, m, n_sms, s);
    if (rows <= 16)
        return launch_nq<16>(a, rt, m, n_sms, s);
    if (rows <= kWeightsFewRows)
        return launch_nq<32>(a, rt, m, n_sms, s);
    return launch_window(a, rt, m, n_sms, s);
}

}  // namespace kvr
