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
// First a unit's kept rows: the threshold weight by a radix select over
// order-preserving integer keys, then the rows at or above it in order, a chain
// of short passes bound by their latency.  Then the kept rows are gathered: an
// HBM stream like the stitch.  With many units or few rows both in one kernel
// (k_evict_unit), else a kernel each (k_evict_select, k_evict_move).
// Measured (bf16, head_dim 128): 4,608 units of 1,044 to 1,344 rows to 512: 370 us, of
// which 362 are the rows' and weights' bytes at the copy rate; 256 units of
// 33,504 rows to 4,096: 52 us + 167 us (6.6 TB/s); 112 units of 2,656 rows to
// 1,024: 9 us + 19 us (6.3 TB/s).
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "kvr_internal.cuh"

namespace kvr {

namespace {

constexpr int kMoveThreads = 256;
constexpr int kSelThreads = 1024;
// CTAs per SM that the registers must leave room for (a bf16 row of 128: 82
// registers, two CTAs, 241 us a call for 256 units of 33,504 rows; three 219,
// four 233)
template <typename T, int D>
constexpr int kMoveCtas = sizeof(T) * D > 256 ? 2 : 3;   // (fp32 rows of 128 need 126 registers)
__host__ __device__ constexpr int evict_chunks(int keep) { return keep > 0 ? (keep + kEvictChunk - 1) / kEvictChunk : 1; }

// Integer key in the order of the weights: NaN lowest, then -inf .. +inf, both
// zeros alike.  Two more values: kNoRow below all of them, for places past the
// rows, and kAlways above, for rows that stay whatever they weigh.
constexpr uint32_t kNoRow = 0u, kNanKey = 1u, kMaxKey = 0xff800000u, kAlways = 0xffffffffu;
__device__ __forceinline__ uint32_t weight_key(uint32_t bits)
{
    if ((bits & 0x7fffffffu) > 0x7f800000u)
        return kNanKey;
    const uint32_t u = bits == 0x80000000u ? 0u : bits;
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

// One CTA of TH threads per (request, unit).  The threshold is found 11, 11 and
// 10 bits at a time: a histogram of the candidates' next digit, and the digit in
// which the k-th largest falls (11 bits: a float's exponent and two bits of its
// fraction, so that heavy-tailed weights already spread over many bins).  Once
// at most kRankMax candidates are left, each counts the candidates before it,
// (weight, then lower row) deciding.  With many rows the shared-memory atomics
// of the first histogram dominate: there an eighth of the rows is counted first,
// and then only the rows in the digits that the k-th largest can lie in.
// Warp w owns rows [32 R' w, 32 R' (w + 1)), R' = ceil(n / TH); it counts what it
// keeps and writes its rows behind the warps before it.  The rows' keys are read
// once, into shared memory (kept in registers, the passes over them were
// unrolled code that runs once, at the speed of instruction fetches: 65 us
// against 52 for 256 units of 33,504 rows); a unit of more rows than fit there
// reads them in every pass.
constexpr int kRankMax = 256;
constexpr int kSelSmemRows = 48 * 1024;   // 192 KB

template <int TH, bool kSmem>
__device__ __forceinline__ void select_rows(const EvictArgs &a, const DevEvict rq, int lh)
{
    constexpr int NW = TH / 32, BPT = 2048 / TH;   // warps, bins of a thread
    int32_t *kept = a.kept + rq.kept0 + (int64_t)lh * rq.keep;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (rq.keep == rq.n) {
        for (int i = threadIdx.x; i < rq.n; i += TH)
            kept[i] = i;
        return;
    }
    const float *w = a.weights + rq.src_row0 + (int64_t)lh * rq.src_cap;
    const int lo = a.n_first, hi = rq.n - a.n_recent;   // rows that compete
    const int k = rq.keep - a.n_first - a.n_recent;     // how many of them stay
    const int n_r = (rq.n + TH - 1) / TH, row0 = warp * 32 * n_r + lane;

    __shared__ int hist[2048];
    __shared__ int s_warp[NW], s_eq[NW];
    __shared__ int s_found[3];                  // digit, rank in it (1 based), candidates in it
    __shared__ int s_n;
    __shared__ uint2 s_cand[kRankMax];          // (key, row)
    __shared__ uint2 s_last;                    // the last candidate that stays
    auto bits_of = [&](int r) -> uint32_t {
        const int i = row0 + 32 * r;
        return i < rq.n ? __float_as_uint(w[i]) : 0u;
    };
    auto key_of = [&](int r, uint32_t bits) -> uint32_t {
        const int i = row0 + 32 * r;
        return i >= rq.n ? kNoRow : i < lo || i >= hi ? kAlways : weight_key(bits);
    };
    // keys: [warp][r / 4][lane] of four rows r .. r + 3 of the lane
    extern __shared__ uint4 keys[];
    const int n_q = (n_r + 3) / 4;
    uint4 *mine = keys + warp * 32 * n_q + lane;
    auto quad_of = [&](int q) -> uint4 {   // from global memory
        uint32_t u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            u[e] = 4 * q + e < n_r ? bits_of(4 * q + e) : 0u;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            u[e] = 4 * q + e < n_r ? key_of(4 * q + e, u[e]) : kNoRow;
        return make_uint4(u[0], u[1], u[2], u[3]);
    };
    if constexpr (kSmem) {
#pragma unroll 4
        for (int q = 0; q < n_q; ++q)   // (sixteen loads in flight)
            mine[32 * q] = quad_of(q);
    }
    // f(row, its key) for every row of the thread, in row order (or every eighth)
    auto each = [&](auto &&f) {
#pragma unroll 2
        for (int q = 0; q < n_q; ++q) {
            const uint4 x = kSmem ? mine[32 * q] : quad_of(q);
            const int i = row0 + 128 * q;
            f(i, x.x);
            f(i + 32, x.y);
            f(i + 64, x.z);
            f(i + 96, x.w);
        }
    };
    auto each8 = [&](auto &&f) {
        for (int q = 0; q < n_q; q += 2)
            f(row0 + 128 * q, kSmem ? mine[32 * q].x : quad_of(q).x);
    };
    auto clear = [&] {
        __syncthreads();
        for (int i = threadIdx.x; i < 2048; i += TH)
            hist[i] = 0;
        if (threadIdx.x == 0)
            s_found[0] = -1;
        __syncthreads();
    };
    auto block_sum_before = [&](int v, int &total) -> int {   // sum over the threads before this one
        int incl = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += u;
        }
        if (lane == 31)
            s_warp[warp] = incl;
        __syncthreads();
        int before = 0;
        total = 0;
        for (int x = 0; x < NW; ++x) {
            before += x < warp ? s_warp[x] : 0;
            total += s_warp[x];
        }
        __syncthreads();
        return before + incl - v;
    };
    // The histogram's digit in which the `rank`-th largest falls (-1: none), from
    // the largest digit down; thread t holds digits 2047 - BPT t and below.
    auto find = [&](int above, int total, int rank) -> int {
        const int d0 = 2047 - BPT * (int)threadIdx.x;
        int run = above;
#pragma unroll
        for (int e = 0; e < BPT; ++e) {
            const int c = hist[d0 - e];
            if (run < rank && rank <= run + c) {
                s_found[0] = d0 - e;
                s_found[1] = rank - run;
                s_found[2] = c;
            }
            run += c;
        }
        __syncthreads();
        return s_found[0];
    };
    auto bins_before = [&](int &total) -> int {
        int sum = 0;
#pragma unroll
        for (int e = 0; e < BPT; ++e)
            sum += hist[2047 - BPT * (int)threadIdx.x - e];
        return block_sum_before(sum, total);
    };

    uint32_t prefix = 0;   // the threshold's leading digits
    int left = k;          // how many of the rows with those digits stay
    bool ranked = false;
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        constexpr int kShift[3] = {21, 10, 0};
        const int shift = kShift[pass], above_bits = pass == 0 ? 31 : kShift[pass == 0 ? 0 : pass - 1];
        if (k == 0 || ranked)
            break;
        int d_lo = 0, d_hi = 2047, above = 0, total = 0;
        bool whole = true;
        if (pass == 0 && n_r >= 8) {
            clear();
            each8([&](int, uint32_t x) {
                if (x - 1u < kMaxKey)   // kNanKey .. kMaxKey
                    atomicAdd(&hist[x >> 21], 1);
            });
            __syncthreads();
            const int before = bins_before(total);
            // the sample's rank, and six standard deviations on both sides
            const float est = (float)k * (float)total / (float)(hi - lo), dev = 6.f * sqrtf((float)total) * 0.5f + 2.f;
            const int r_hi = (int)(est - dev), r_lo = (int)(est + dev);
            if (r_hi >= 1)
                d_hi = find(before, total, r_hi);
            __syncthreads();
            if (r_lo <= total)
                d_lo = find(before, total, r_lo);
            whole = d_lo == 0 && d_hi == 2047;
        }
        for (;;) {
            clear();
            int n_above = 0;
            if (pass == 0) {
                const uint32_t k_lo = max(kNanKey, (uint32_t)d_lo << 21), k_hi = min(kMaxKey, ((uint32_t)d_hi << 21) | 0x1fffffu);
                each([&](int, uint32_t x) {
                    n_above += x > k_hi;
                    if (x - k_lo <= k_hi - k_lo)
                        atomicAdd(&hist[x >> 21], 1);
                });
            } else {
                each([&](int, uint32_t x) {
                    if (x != kNoRow && (x >> above_bits) == (prefix >> above_bits))
                        atomicAdd(&hist[(x >> shift) & 2047], 1);
                });
            }
            __syncthreads();
            if (!whole) {
                block_sum_before(n_above, above);
                above -= a.n_first + a.n_recent;   // (kAlways is above every digit)
            }
            const int before = bins_before(total);
            if (find(above + before, total, left) >= 0)
                break;
            d_lo = 0;   // outside the sample's digits (they are six deviations wide): count all
            d_hi = 2047;
            whole = true;
            above = 0;
        }
        prefix |= (uint32_t)s_found[0] << shift;
        left = s_found[1];
        const int n_cand = s_found[2];
        if (n_cand <= kRankMax) {
            // collected, with each warp's count of the keys above the digit; then the
            // ones among the candidates that stay are added to their warps' counts
            ranked = true;
            if (threadIdx.x == 0)
                s_n = 0;
            __syncthreads();
            const uint32_t digit = prefix >> shift;
            int n_gt = 0;
            each([&](int i, uint32_t x) {
                const uint32_t d = x >> shift;
                n_gt += d > digit;
                if (d == digit && x != kNoRow) {
                    const int c = atomicAdd(&s_n, 1);
                    if (c < kRankMax)
                        s_cand[c] = make_uint2(x, (uint32_t)i);
                }
            });
            n_gt = __reduce_add_sync(0xffffffffu, n_gt);
            if (lane == 0)
                s_warp[warp] = n_gt;
            __syncthreads();
            for (int c = threadIdx.x; c < n_cand; c += TH) {
                const uint2 me = s_cand[c];
                int rank = 0;
                for (int o = 0; o < n_cand; ++o) {
                    const uint2 v = s_cand[o];
                    rank += v.x > me.x || (v.x == me.x && v.y < me.y);
                }
                if (rank < left)
                    atomicAdd(&s_warp[(int)me.y / (32 * n_r)], 1);
                if (rank == left - 1)
                    s_last = me;
            }
            __syncthreads();
        }
    }
    // Kept: keys above the threshold (kAlways among them); of the keys equal to it
    // those up to row s_last.y (ranked), or the `left` lowest rows
    const uint32_t thr = k == 0 ? kAlways - 1u : ranked ? s_last.x : prefix;
    const int last_row = ranked ? (int)s_last.y : -1;
    const bool ties = k > 0 && !ranked;
    if (!ranked) {
        int n_gt = 0, n_eq = 0;
        each([&](int, uint32_t x) {
            n_gt += x > thr;
            n_eq += x == thr;
        });
        n_gt = __reduce_add_sync(0xffffffffu, n_gt);
        n_eq = __reduce_add_sync(0xffffffffu, n_eq);
        __syncthreads();
        if (lane == 0) {
            s_warp[warp] = n_gt;
            s_eq[warp] = ties ? n_eq : 0;
        }
        __syncthreads();
    }
    int gt_before = 0, eq_before = 0;
    for (int x = 0; x < warp; ++x) {
        gt_before += s_warp[x];
        eq_before += ranked ? 0 : s_eq[x];
    }
    const unsigned below = (1u << lane) - 1u;
    if (!ties) {
        each([&](int i, uint32_t x) {
            const bool gt = x > thr || (x == thr && i <= last_row);
            const unsigned bg = __ballot_sync(0xffffffffu, gt);
            if (gt)
                kept[gt_before + __popc(bg & below)] = i;
            gt_before += __popc(bg);
        });
    } else {
        each([&](int i, uint32_t x) {
            const bool gt = x > thr, eq = x == thr;
            const unsigned bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
            const int g = gt_before + __popc(bg & below), e = eq_before + __popc(be & below);
            if (gt || (eq && e < left))
                kept[g + min(e, left)] = i;
            gt_before += __popc(bg);
            eq_before += __popc(be);
        });
    }
}

template <bool kSmem>
__global__ void __launch_bounds__(kSelThreads, 1)
    k_evict_select(const __grid_constant__ EvictArgs a, const __grid_constant__ EvictTable rt)
{
    pdl_wait_prerequisites();
    pdl_launch_dependents();   // (the move kernel waits for this grid)
    const int b = (int)(blockIdx.x / (unsigned)a.units);
    select_rows<kSelThreads, kSmem>(a, (a.reqs ? a.reqs : rt.reqs)[b], (int)(blockIdx.x % (unsigned)a.units));
}

// Rows c_first * kEvictChunk .. of unit lh: pieces of kEvictChunk kept rows.  TPR threads a row, thread j
// holding 16-byte vector j of each row half (so that both halves of a RoPE
// pair are in one thread).  A bf16 key's angles are computed, not read: a moved
// row's (cos, sin) table row would be 512 bytes beside the 512 of its K and V.
// The turn delta * w_i / 2 pi is reduced exactly (an fp32 product with the
// frequency in two words), and sin and cos of the rest are good to 2^-20, far
// below the bf16 result's 2^-9.  In place, a CTA walks its unit's pieces in
// order: a piece's sources lie at or behind its own rows, so once the piece is
// read (barrier), writing it only overwrites rows that were read before.
// `wait` is called before the kept rows are read.
template <typename T, int D, typename Wait>
__device__ __forceinline__ void move_rows(const EvictArgs &a, const DevEvict rq, int lh, int c_first, int c_end, Wait &&wait)
{
    constexpr int E = RowVec<T>::E, H2 = D / 2, TPR = H2 / E, RPP = kMoveThreads / TPR;
    constexpr int NR = (kEvictChunk + RPP - 1) / RPP;   // rows of a thread
    const int32_t *kept = a.kept + rq.kept0 + (int64_t)lh * rq.keep;
    const int64_t src0 = rq.src_row0 + (int64_t)lh * rq.src_cap, dst0 = rq.dst_row0 + (int64_t)lh * rq.dst_cap;
    const T *sk = static_cast<const T *>(a.cache_k) + src0 * D, *sv = static_cast<const T *>(a.cache_v) + src0 * D;
    T *dk = static_cast<T *>(a.dst_k) + dst0 * D, *dv = static_cast<T *>(a.dst_v) + dst0 * D;
    const float *sw = a.weights + src0;
    float *dw = a.dst_weights ? a.dst_weights + dst0 : nullptr;
    const int j = threadIdx.x % TPR, rr = threadIdx.x / TPR;
    float f_hi[E], f_lo[E];   // the thread's pairs' frequencies in turns
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float2 f = __ldg(a.rope_turns + rope_pair(a.interleaved, D, E, j, e));
            f_hi[e] = f.x;
            f_lo[e] = f.y;
        }
    }
    wait();
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
                    if constexpr (sizeof(T) == 2) {
                        const float fd = (float)delta, q = rintf(fd * f_hi[e]);
                        const float turn = fmaf(fd, f_lo[e], fmaf(fd, f_hi[e], -q));   // in [-1/2, 1/2], to 2^-24
                        __sincosf(turn * 6.283185307179586f, &sn[e], &cs[e]);
                    } else {
                        const float2 r = rope_cs(a.rope, H2, delta, rope_pair(a.interleaved, D, E, j, e));
                        cs[e] = r.x;
                        sn[e] = r.y;
                    }
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
    if (dw && c_end == evict_chunks(rq.keep)) {
        if (a.in_place)
            __syncthreads();
        for (int i = rq.keep + (int)threadIdx.x; i < rq.dst_cap; i += kMoveThreads)
            dw[i] = 0.f;
    }
}

// To another block, every piece is a CTA; in place, every unit.
template <typename T, int D>
__global__ void __launch_bounds__(kMoveThreads, kMoveCtas<T, D>)
    k_evict_move(const __grid_constant__ EvictArgs a, const __grid_constant__ EvictTable rt)
{
    const DevEvict *reqs = a.reqs ? a.reqs : rt.reqs;
    if (a.reqs)
        pdl_wait_prerequisites();   // (an uploaded table: promised to a grid that waited itself)
    int b, lh, c_first, c_end;
    if (a.in_place) {
        b = (int)(blockIdx.x / (unsigned)a.units);
        lh = (int)(blockIdx.x % (unsigned)a.units);
        c_first = 0;
        c_end = evict_chunks(reqs[b].keep);
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
        const int n_c = evict_chunks(reqs[b].keep);
        const int local = (int)blockIdx.x - reqs[b].chunk0;
        lh = local / n_c;
        c_first = local - lh * n_c;
        c_end = c_first + 1;
    }
    move_rows<T, D>(a, reqs[b], lh, c_first, c_end, [] { pdl_wait_prerequisites(); });
}

// Both in one: a CTA of 256 threads selects a unit's rows and moves them.  With
// several units per SM one's selection, a chain of short dependent steps,
// overlaps the others' traffic.
template <typename T, int D>
__global__ void __launch_bounds__(kMoveThreads, kMoveCtas<T, D>)
    k_evict_unit(const __grid_constant__ EvictArgs a, const __grid_constant__ EvictTable rt)
{
    pdl_wait_prerequisites();
    const int b = (int)(blockIdx.x / (unsigned)a.units), lh = (int)(blockIdx.x % (unsigned)a.units);
    const DevEvict rq = (a.reqs ? a.reqs : rt.reqs)[b];
    select_rows<kMoveThreads, true>(a, rq, lh);
    move_rows<T, D>(a, rq, lh, 0, evict_chunks(rq.keep), [] { __syncthreads(); });
}

cudaError_t launch_evict(const EvictArgs &a, const EvictTable &rt, int dtype, int head_dim, int n_sms, cudaStream_t s)
{
    const int64_t ctas = (int64_t)a.n_reqs * a.units;
    const int64_t move = a.in_place ? ctas : a.n_chunks;
    if (ctas > 0x7fffffff || move > 0x7fffffff)
        return cudaErrorInvalidValue;
    using Kernel = void (*)(const EvictArgs, const EvictTable);
    auto pick = [&](Kernel b128, Kernel b64, Kernel f128, Kernel f64) -> Kernel {
        if (head_dim != 128 && head_dim != 64)
            return nullptr;
        return dtype == KVR_DTYPE_BF16 ? (head_dim == 128 ? b128 : b64) : (head_dim == 128 ? f128 : f64);
    };
    auto smem_rows = [&](int threads) { return (a.max_n + 4 * threads - 1) / (4 * threads) * 4 * threads; };   // keys there
    // One kernel where units' keys leave room for three CTAs per SM and a CTA's rows
    // do not last beyond the others': any with two units per SM, 1,024 rows with one,
    // 256 with fewer.  4,608 units of up to 1,344 rows to 512: 370 us a call, 531 in
    // two kernels; 224 units, 300 to 150: 8.9 against 16.0, 1,300 to 512: 26 against
    // 31, 2,600 to 1,024: alike; 112 units, 300 to 150: 6.8 against 9.2, 650 to 450:
    // 16.4 against 15.1, 2,600 to 1,024: 37 against 27.
    const int most = ctas >= 2 * (int64_t)n_sms ? a.max_n : ctas >= n_sms ? 1024 : 256;
    if (a.max_n <= 24 * 256 && a.max_keep <= most) {
        const Kernel k = pick(k_evict_unit<__nv_bfloat16, 128>, k_evict_unit<__nv_bfloat16, 64>, k_evict_unit<float, 128>,
                              k_evict_unit<float, 64>);
        if (!k)
            return cudaErrorInvalidValue;
        return launch_pdl(k, ctas, kMoveThreads, smem_rows(kMoveThreads) * 4, true, s, a, rt);
    }
    const int rows = smem_rows(kSelThreads);
    const bool smem = rows <= kSelSmemRows;
    static std::atomic<bool> attr_set[64] = {};   // per device (host threads may race: same value)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev >= 64 || !attr_set[dev].load(std::memory_order_acquire)) {
        if ((e = cudaFuncSetAttribute(k_evict_select<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelSmemRows * 4)) !=
            cudaSuccess)
            return e;
        if (dev < 64)
            attr_set[dev].store(true, std::memory_order_release);
    }
    const Kernel k = pick(k_evict_move<__nv_bfloat16, 128>, k_evict_move<__nv_bfloat16, 64>, k_evict_move<float, 128>,
                          k_evict_move<float, 64>);
    if (!k)
        return cudaErrorInvalidValue;
    e = launch_pdl(smem ? k_evict_select<true> : k_evict_select<false>, ctas, kSelThreads, smem ? rows * 4 : 0, true, s, a, rt);
    return e == cudaSuccess ? launch_pdl(k, move, kMoveThreads, 0, true, s, a, rt) : e;
}

// w_i / 2 pi in two floats (value and what it leaves), pairs 0 .. half - 1.
__global__ void k_rope_turns(float2 *turns, int half, double theta)
{
    const int i = threadIdx.x;
    if (i < half) {
        const double f = pow(theta, -(double)i / (double)half) / 6.283185307179586476925286766559;
        turns[i] = make_float2((float)f, (float)(f - (double)(float)f));
    }
}

cudaError_t launch_rope_turns(float2 *turns, int head_dim, double theta, cudaStream_t s)
{
    k_rope_turns<<<1, 64, 0, s>>>(turns, head_dim / 2, theta);
    return cudaGetLastError();
}

}  // namespace kvr
