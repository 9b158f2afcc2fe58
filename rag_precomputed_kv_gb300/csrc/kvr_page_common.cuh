// kvr_page_common.cuh -- what the kernels of the paged cache share: page
// look-up, which rows a query sees, and the packed rows' layout.
//
// A packed block holds kPackRows = 32 rows of one (layer, kv-head), 16 at a time:
// 1,024 bytes of the keys' 4-bit codes, 128 of their bf16 scales, then the values'.
// A value is scale * (nibble - 8).  Scales lie [n][rows n, n + 8][group of 32 dims]
// (n = 0..7).  Codes lie as the operands of mma.sync m16n8k16 want them, 512 bytes
// for 8 rows, 16 bytes for each lane 4 n + c (c = 0..3), one word per group g:
//   keys    lane 4 n + c: row n, dims 32 g + 8 c + 0..7; nibble m holds the dim
//           2 m, nibble m + 4 the dim 2 m + 1 (m = 0..3): a shift by 4 m and a
//           mask leave two neighbouring dims in the two halves of the word.
//   values  lane 4 n + c: nibbles t = 0..3 row 2 c, nibbles 4 + t row 2 c + 1, dim
//           32 g + 8 t + n: a shift by 4 t and a mask leave two neighbouring
//           rows' values of one dim.
#pragma once

#include <cuda_bf16.h>

#include "kvr_internal.cuh"

namespace kvr {
namespace page {

// The page of a row (a power of two of rows without a division: 33,280 packed rows, 256
// units, 286 -> 273 us).
__device__ __forceinline__ int page_of(const PageArgs &a, int row) { return a.g.shift >= 0 ? row >> a.g.shift : row / a.g.rows; }
__device__ __forceinline__ int32_t page_id(const DevPageReq &r, const int32_t *ids, int pg)
{
    return ids[pg + (pg < r.few ? r.off[0] : r.off[1])];
}
__device__ __forceinline__ int32_t packed_id(const DevPageReq &r, const int32_t *ids, int pg)
{
    return ids[pg + (pg < r.pfew ? r.poff[0] : r.poff[1])];
}

// The last request whose first token is <= t and that has tokens behind it.
__device__ __forceinline__ int request_of(const DevPageReq *reqs, int n, int t)
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (reqs[mid].q_off <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// Rows that the query at position p sees: j < hi and (j >= lo or j < few).
struct Sees {
    int hi, lo, few;
    __device__ __forceinline__ bool operator()(int j) const { return j < hi && (j >= lo || j < few); }
};
__device__ __forceinline__ Sees sees(const PageArgs &a, const DevPageReq &r, int p)
{
    Sees s;
    s.hi = min(r.kv_len, p + 1);
    s.lo = a.window > 0 ? max(0, p - a.window + 1) : 0;
    s.few = min(a.n_first, s.lo);
    return s;
}

// Offsets in a block: the codes of rows 8 i .. 8 i + 7, the four scales of row r; of the
// keys (part 0) or the values (1).
__device__ __forceinline__ int codes_at(int i, int part) { return (i >> 1) * kPackStep + part * kPackPart + (i & 1) * 512; }
__device__ __forceinline__ int scales_at(int r, int part)
{
    return (r >> 4) * kPackStep + part * kPackPart + 1024 + (r & 7) * 16 + (r & 8);
}

// Rows that some query of a request sees.
__device__ __forceinline__ Sees sees_any(const PageArgs &a, const DevPageReq &r)
{
    Sees s;
    s.hi = min(r.kv_len, r.pos0 + r.q_len);
    s.lo = min(s.hi, a.window > 0 ? max(0, r.pos0 - a.window + 1) : 0);
    s.few = min(a.n_first, s.lo);
    return s;
}

// The 128-row tiles of a request that hold packed rows are restored: its first `first` ones and
// those from `win` up to `end`, one behind the other.
struct RestTiles {
    int first, win, end;
    __device__ __forceinline__ int count() const { return first + max(0, end - win); }
    __device__ __forceinline__ int tile(int i) const { return i < first ? i : win + i - first; }
    __device__ __forceinline__ int place(int t) const { return t < first ? t : first + t - win; }
};
__host__ __device__ __forceinline__ RestTiles rest_tiles(int hi, int lo, int few, int body)
{
    RestTiles r;
    const int e = hi < body ? hi : body, a = (few + 127) / 128;
    r.end = (e + 127) / 128;
    r.first = a < r.end ? a : r.end;
    r.win = a > lo / 128 ? a : lo / 128;
    return r;
}

// Byte offset of packed row block `row / 32` in the packed pages.
__device__ __forceinline__ int64_t packed_block(const PageArgs &a, const DevPageReq &r, const int32_t *ids, int lh, int row)
{
    const int pg = page_of(a, row), in = row - pg * a.g.rows;
    return (int64_t)packed_id(r, ids, pg) * a.g.packed_page + ((int64_t)lh * (a.g.rows / kPackRows) + in / kPackRows) * kPackBytes;
}

// 8x8 nibbles across the 8 lanes of an octet: lane i's nibble j becomes lane j's
// nibble i.
__device__ __forceinline__ uint32_t transpose_nibbles(uint32_t w, int lane)
{
#pragma unroll
    for (int b = 4; b >= 1; b >>= 1) {
        // the halves that stay, and that change places with lane ^ b
        const uint32_t mask = b == 4 ? 0x0000ffffu : b == 2 ? 0x00ff00ffu : 0x0f0f0f0fu;
        const uint32_t other = __shfl_xor_sync(0xffffffffu, w, b);
        w = (lane & b) ? ((w & ~mask) | ((other >> (4 * b)) & mask)) : ((w & mask) | ((other << (4 * b)) & ~mask));
    }
    return w;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t s) { return __byte_perm(a, b, s); }
__device__ __forceinline__ uint32_t hmul2_bf16(uint32_t a, uint32_t b)
{
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}
// Nibbles 0 and 4 of w, less 8, as a bf16 pair (128 + nibble less 136: exact).
__device__ __forceinline__ uint32_t code_pair(uint32_t w)
{
    const uint32_t x = (w & 0x000f000fu) | 0x43004300u, c = 0x43084308u;
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&x), *reinterpret_cast<const __nv_bfloat162 *>(&c));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Eight values of a packed word (dims 32 g + 8 c .. of the lane's row), times their scale
// (in both halves of s), each rounded once.  part 1: a value word, of the lane that its
// octet's transposition puts in this lane's place.
__device__ __forceinline__ uint4 restore8(uint32_t w, int part, uint32_t s, int lane)
{
    uint32_t v[4];
    if (part) {
        w = transpose_nibbles(w, lane);   // dims in order
#pragma unroll
        for (int m = 0; m < 4; ++m)       // (nibbles 2 m and 2 m + 1 into bytes 0 and 2)
            v[m] = code_pair(prmt(w, w >> 4, 0x0400u + 0x0101u * (uint32_t)m));
    } else {
#pragma unroll
        for (int m = 0; m < 4; ++m)
            v[m] = code_pair(w >> (4 * m));
    }
    return make_uint4(hmul2_bf16(v[0], s), hmul2_bf16(v[1], s), hmul2_bf16(v[2], s), hmul2_bf16(v[3], s));
}

}  // namespace page
}  // namespace kvr
