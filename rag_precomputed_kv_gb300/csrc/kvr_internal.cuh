// kvr_internal.cuh -- types shared by the libkvr translation units.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <utility>

#include "../../include/kvr.h"

#ifdef __CUDACC__
#include <cuda_bf16.h>
#endif

namespace kvr {

// RoPE tables: angle(n, i) = n * theta^(-2i/D) for n in [0, 2^24) is split as
// n = hi * 4096 + lo; the table holds (cos, sin) of hi * 4096 * w_i
// (rows 0..4095) and of lo * w_i (rows 4096..8191), each computed in double
// precision and rounded to float.  One complex product in float recombines
// them: the angle-addition identity, with error of a few float ulps for
// every position (a float product n * w_i would be off by up to ~2e-3 rad at
// n ~ 3e4).
constexpr int kRopeSplit = 4096;
constexpr int kMaxPosition = kRopeSplit * kRopeSplit;  // 2^24

#ifdef __CUDACC__
// Programmatic dependent launch: let the next kernel of the stream (launched
// with programmatic serialization) start its grid now / wait until the
// previous kernel of the stream has completed and its writes are visible.
__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait_prerequisites() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// (cos, sin) of pos * w_i for |pos| < 2^24 from the two table halves (angle
// addition, one complex product in float); a negative pos is the conjugate.
// Below 2^12 the high half's entry is row 0, exactly (1, 0): the product is
// the low entry itself, bit for bit, and only that one is read.
__device__ __forceinline__ float2 rope_cs(const float2 *__restrict__ tab, int half, int pos, int i)
{
    const int a = pos < 0 ? -pos : pos;
    const float2 l = __ldg(tab + (kRopeSplit + (a & (kRopeSplit - 1))) * half + i);
    float c = l.x, s = l.y;
    if (a >= kRopeSplit) {
        const float2 h = __ldg(tab + (a >> 12) * half + i);
        c = fmaf(h.x, l.x, -h.y * l.y);
        s = fmaf(h.y, l.x, h.x * l.y);
    }
    return make_float2(c, pos < 0 ? -s : s);
}

// RoPE rotation of 8 bf16 pairs: lo holds elements [8j, 8j+8) of a row, hi
// their partners [D/2 + 8j, ...); (c, s) of each pair.  The stitch kernel's
// key re-rotation for bf16 caches.
// Per pair: x' = fma(x, c, -(y s)), y' = fma(x, s, y c), rounded once to bf16;
// computed two lanes at a time with the packed fp32 instructions (each lane
// is the IEEE operation of the scalar form).
__device__ __forceinline__ void rotate_bf16x8(uint4 &lo, uint4 &hi, const float *c, const float *s)
{
    uint32_t *pl = reinterpret_cast<uint32_t *>(&lo);
    uint32_t *ph = reinterpret_cast<uint32_t *>(&hi);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        // bf16 pair -> two fp32 lanes (a bf16 is the high half of its fp32)
        const uint64_t x = ((uint64_t)(pl[w] & 0xffff0000u) << 32) | (uint64_t)(pl[w] << 16);
        const uint64_t y = ((uint64_t)(ph[w] & 0xffff0000u) << 32) | (uint64_t)(ph[w] << 16);
        const uint64_t cc = ((uint64_t)__float_as_uint(c[2 * w + 1]) << 32) | __float_as_uint(c[2 * w]);
        const uint64_t ns = ((uint64_t)__float_as_uint(-s[2 * w + 1]) << 32) | __float_as_uint(-s[2 * w]);
        const uint64_t ss = ((uint64_t)__float_as_uint(s[2 * w + 1]) << 32) | __float_as_uint(s[2 * w]);
        uint64_t ys, yc, xo, yo;
        asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(ys) : "l"(y), "l"(ns));
        asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(yc) : "l"(y), "l"(cc));
        asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(xo) : "l"(x), "l"(cc), "l"(ys));
        asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(yo) : "l"(x), "l"(ss), "l"(yc));
        __nv_bfloat162 xb = __floats2bfloat162_rn(__uint_as_float((uint32_t)xo), __uint_as_float((uint32_t)(xo >> 32)));
        __nv_bfloat162 yb = __floats2bfloat162_rn(__uint_as_float((uint32_t)yo), __uint_as_float((uint32_t)(yo >> 32)));
        pl[w] = *reinterpret_cast<uint32_t *>(&xb);
        ph[w] = *reinterpret_cast<uint32_t *>(&yb);
    }
}

// The same rotation for the interleaved pairing: every bf16 word of lo and
// hi is a pair (x_2i, x_2i+1); c[w], s[w] belong to lo's word w and c[4 + w],
// s[4 + w] to hi's.
__device__ __forceinline__ void rotate_bf16x8_il(uint4 &lo, uint4 &hi, const float *c, const float *s)
{
    uint32_t *pw[2] = {reinterpret_cast<uint32_t *>(&lo), reinterpret_cast<uint32_t *>(&hi)};
#pragma unroll
    for (int v = 0; v < 2; ++v) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float2 xy = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&pw[v][w]));
            const float cc = c[4 * v + w], ss = s[4 * v + w];
            __nv_bfloat162 o = __floats2bfloat162_rn(fmaf(xy.x, cc, -xy.y * ss), fmaf(xy.x, ss, xy.y * cc));
            pw[v][w] = *reinterpret_cast<uint32_t *>(&o);
        }
    }
}

// Pair index of the e-th (cos, sin) of a thread that owns 16-byte chunk j of
// both row halves (E elements per chunk, head dim D): half-split pairs are
// elements (jE + e, D/2 + jE + e); interleaved pairs are whole inside a
// chunk, E/2 of them in the chunk of each half.
__device__ __forceinline__ int rope_pair(bool interleaved, int D, int E, int j, int e)
{
    if (!interleaved)
        return j * E + e;
    return e < E / 2 ? (E / 2) * j + e : D / 4 + (E / 2) * j + (e - E / 2);
}
#endif

// Device copy of one span (48 bytes).
struct alignas(16) DevSpan {
    int64_t dst_row0;  // first row of the request's cache block, in head_dim rows
    int64_t flat0;     // index of the span's first token in the flat pos / src maps
    int32_t src;       // pool entry, or KVR_SRC_LOCAL | local index
    int32_t start;     // first source token
    int32_t len;       // tokens
    int32_t row;       // first stitched row inside the request's block
    int32_t delta;     // rotation applied to the keys (positions)
    int32_t pos0;      // position id of the first token
    int32_t cap;       // rows per (layer, kv-head) block of the request
    int32_t dstep;     // 0: source keys carry their source positions (rotate all
                       //    tokens by delta); 1: source keys are un-rotated
                       //    (token t is rotated by delta + t)
};

// Device copy of one request-local source.
struct alignas(16) DevLocal {
    const void *k;
    const void *v;
    int64_t s_layer, s_head, s_tok;
    int64_t len;
};

// Per-request data for the attention kernels (48 bytes).  On the tensor-core
// path the table is in schedule order (longest prefix first) and unit0 is the
// request's first work unit; elsewhere it is in request order.
struct alignas(16) DevReq {
    int64_t cache_row0;  // cache_offsets[b] * L * H_kv
    int32_t cap;         // R_b
    int32_t prefix;      // P_b
    int32_t q_off;       // first query token (token axis of q / out)
    int32_t q_len;       // Lq_b
    int32_t unit0;       // first (layer, kv-head, 256-row block) unit (tensor-core path)
    int32_t span0;       // first non-empty span of this request (values-gathering attention)
    int32_t span_end;    // one past its last
    int32_t flags;       // kReqValuesTma (values-gathering attention)
    int32_t pad_[2];
};
static_assert(sizeof(DevReq) == 48, "request table layout");
// DevReq::flags: the values-gathering attention loads this request's prefix
// value tiles through TMA box loads (its spans are long and all from a
// contiguous pool) rather than with the gather warps' copies
constexpr int32_t kReqValuesTma = 1;

// Device error word codes (first error wins).  kDevBadInput: an attention
// row's softmax denominator came out non-finite or zero (a NaN or infinity in
// the query heads or the keys it saw); the row's output is written as computed.
enum : int { kDevOk = 0, kDevTimeout = 1, kDevBadInput = 2 };

// Records `msg` as this host thread's last error (kvr_last_error) and
// returns `st`; allocates nothing.
kvr_status record_error(kvr_status st, const char *msg);

struct AssembleArgs {
    const DevSpan *spans;
    const DevLocal *locals;
    const float2 *rope;
    const void *pool_k;
    const void *pool_v;
    int64_t ps_entry, ps_layer, ps_head, ps_tok;
    void *cache_k;
    void *cache_v;
    int32_t *pos_ids;
    int32_t *src_map;
    int32_t n_layers, n_heads;  // kv heads
    int32_t upc;                // (layer, head) units per CTA
    int32_t interleaved;        // RoPE pairs (x_2i, x_2i+1)
    // a slice of the (layer, kv-head) units, [lh_begin, lh_begin + lh_count)
    // (lh_count 0: all of them); the position ids and source map are written
    // with the slice that starts at unit 0
    int32_t lh_begin, lh_count;
    // > 0: at most this many CTAs, each looping over (span, unit group)
    // pieces (the stitch then leaves the other SMs to a concurrent kernel)
    int32_t max_ctas;
    int32_t n_spans;            // set by launch_assemble
    int32_t keys_only;          // stitch K (and the maps) only; V is gathered by the attention
};

// Span / local-source tables passed inside the kernel parameters (no upload)
// when a call has at most kInlineEntries of each.
constexpr int kInlineEntries = 64;
struct AssembleTables {
    DevSpan spans[kInlineEntries];
    DevLocal locals[kInlineEntries];
};

// Request table passed inside the attention kernels' parameters when
// batch <= kInlineEntries (AttnArgs::reqs is then NULL).
struct ReqTable {
    DevReq reqs[kInlineEntries];
};

struct AttnArgs {
    const DevReq *reqs;
    int32_t n_reqs;
    const float2 *rope;
    const void *q;              // [L][T][Hq][D]
    const void *cache_k;
    const void *cache_v;
    void *out;                  // [L][T][Hq][D]
    int32_t n_layers, n_q_heads, n_kv_heads;
    int32_t total_q;            // T
    float scale_log2;           // softmax scale * log2(e)
    int *err;
    // tensor-core kernel: units n_full.. (the last wave's, when two halves of
    // each fit one wave) run as two halves of their key range on the two CTAs
    // of a cluster, which merge them; n_full < units requires a launch in
    // two-CTA clusters
    int32_t n_full;
    int32_t interleaved;        // RoPE pairs (x_2i, x_2i+1)
    // tensor-core kernel: a slice of each request's (layer, kv-head) units,
    // [lh_base, lh_base + lh_count) (lh_count 0: all); the request table's
    // unit0 counts lh_count units per 256-row block
    int32_t lh_base, lh_count;
    // tensor-core kernel: the output goes out through TMA tensor stores (the
    // tmap_out parameter), a warp's 32 rows = 32 / G whole tokens of the G
    // query heads of one kv head; set when G is a power of two and `out` is
    // device memory
    int32_t out_tma;
};

struct QueryPrologueArgs {
    const DevReq *reqs;         // NULL: the ReqTable parameter holds the requests
    const float2 *rope;
    const void *q;              // [L][T][Hq][D], not rotated
    const void *kq;             // [L][T][Hkv][D], not rotated
    const void *vq;
    void *cache_k;
    void *cache_v;
    void *q_rot;                // out: [L][Hkv][T][G][D], rotated at P_b + t
    int32_t n_layers, n_q_heads, n_kv_heads;
    int32_t total_q;            // T
    int32_t max_q_len;          // longest query of the batch
    int32_t n_reqs;
    int32_t interleaved;        // RoPE pairs (x_2i, x_2i+1)
};

// A launch whose kernel may set up before the kernel before it is done (it waits
// with pdl_wait_prerequisites); pdl false: a plain one.
template <typename... P, typename... A>
inline cudaError_t launch_pdl(void (*k)(P...), int64_t grid, int block, int smem, bool pdl, cudaStream_t s, A &&...args)
{
    if (grid > 0x7fffffff)
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k, std::forward<A>(args)...);
}

// The same in clusters of c CTAs.
template <typename... P, typename... A>
inline cudaError_t launch_cluster(void (*k)(P...), int64_t grid, int block, int smem, int c, cudaStream_t s, A &&...args)
{
    if (grid > 0x7fffffff)
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)c;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k, std::forward<A>(args)...);
}

// ---- query attention over a prefix shared by a group of requests ----
// Per-request data (64 bytes): the request's own cache block, as DevReq, and
// the prefix block of its group.
struct alignas(16) DevShared {
    int64_t cache_row0;  // own block: cache_offsets[b] * L * H_kv
    int64_t pre_row0;    // prefix block: prefix_offsets[g] * L * H_kv
    int32_t cap;         // own rows per (layer, kv-head) block
    int32_t own;         // own rows that hold data before the call
    int32_t pre_cap;     // rows per (layer, kv-head) block of the prefix
    int32_t pre_len;     // P_g; query token t sits at position P_g + own + t
    int32_t q_off, q_len;
    int32_t group;       // index into the group table (tensor-core path)
    int32_t chunk0;      // the request's first row chunk of a unit (k_shared_own_rows)
    int32_t pad_[4];
};
static_assert(sizeof(DevShared) == 64, "shared-prefix request table layout");
struct SharedTable {
    DevShared reqs[kInlineEntries];
};
struct SharedArgs {
    const DevShared *reqs;      // NULL: the SharedTable parameter
    const float2 *rope;
    const void *q, *kq, *vq;
    const void *prefix_k, *prefix_v;
    void *cache_k, *cache_v;
    void *out;
    int32_t n_reqs;
    int32_t n_layers, n_q_heads, n_kv_heads;
    int32_t total_q;            // T
    float scale_log2;
    int32_t interleaved;
    int *err;
    // tensor-core path: relay[0] holds `call` once a CTA of the prologue has waited for the
    // work before the call, relay[1] once one of the prefix part has waited for the prologue
    uint32_t *relay;
    uint32_t call;              // number of the pool's call, from 1 on
};

// Per-group data (64 bytes) of the tensor-core path: the packed query rows of
// the group's tokens are consecutive, and meet the prefix in blocks of 256.
// The (block, key tile) pairs of a (layer, kv-head) unit are numbered group by
// group; groups without prefix or tokens come last in the table, with nt 0 and
// the unit's number of pairs as w0.
struct alignas(16) DevGroup {
    int64_t pre_row0;    // prefix_offsets[g] * L * H_kv
    int64_t item0;       // the group's first 256-row block of a unit
    int64_t w0;          // the group's first (block, key tile) pair of a unit
    int32_t pre_cap, pre_len;
    int32_t q_off;       // first token
    int32_t rows;        // tokens x G
    int32_t nt;          // 128-key tiles of the prefix
    int32_t mb;          // 256-row blocks
    int32_t pad_[4];
};
static_assert(sizeof(DevGroup) == 64, "group table layout");
struct GroupTable {
    DevGroup groups[kInlineEntries];
};
// Query rows of a request up to which k_shared_own_decode takes its own part, and those
// that one row group of k_shared_own_rows holds.
constexpr int kOwnFewRows = 16, kOwnRowsMax = 64;
// Bytes of one partial result of the prefix part (a block's rows of one CTA:
// 256 x 128 fp32 and 256 maxima and sums).
constexpr int64_t kSharedPartBytes = 256 * 128 * 4 + 256 * 8;
struct SharedPrefixArgs {
    const DevGroup *groups;     // NULL: the GroupTable parameter
    int32_t n_groups;
    int32_t group;              // G
    int32_t total_q;
    int32_t lh_base, lh_count;  // the slice of (layer, kv-head) units of this launch
    int32_t n_ctas;             // stretches that the pairs are cut in
    int64_t unit_pairs, unit_blocks;   // pairs, blocks of one unit
    int64_t total;              // pairs (whole: blocks) of the slice: lh_count times a unit's
    float ratio;                // n_ctas / total
    int32_t run;                // whole: consecutive blocks of a CTA
    float *part;                // (blocks + n_ctas) partial results
    const void *q_rot;          // [L][Hkv][T][G][D], rotated
    float scale_log2;
    int *err;
    uint32_t *relay;            // as in SharedArgs
    uint32_t call;
};
struct SharedTcArgs {
    const SharedArgs *base;
    const SharedTable *reqs;
    const SharedPrefixArgs *prefix;
    const GroupTable *groups;
    // host CUtensorMaps: packed queries and prefix (64 x 128 boxes; the prefix's
    // NULL when nothing is shared), own caches (64 x 32)
    // (whole: 64 x 128)
    const void *tmap_q, *tmap_pk, *tmap_pv, *tmap_k, *tmap_v;
    int32_t n_sms;
    bool whole;                 // the prefix kernel takes whole blocks, and their rows' own keys too
    int32_t few_rows;           // most query rows of a request that k_shared_own_decode takes (0: none)
    int32_t own_per_cta;        // k_shared_own_rows: 64-row groups of a CTA
    int32_t own_chunks;         // its CTAs of a unit (0: no request of more rows than the other takes)
    int32_t max_own_keys;       // the longest own part (own rows and query tokens) of a request of k_shared_own_rows
};

// ---- attention weight per cached key ----
// Query rows of a request up to which it goes to k_key_weights_tc, beyond to
// k_key_weights_window.
constexpr int kWeightsFewRows = 32;
struct WeightsArgs {
    const DevReq *reqs;         // NULL: the ReqTable parameter
    const float2 *rope;
    const void *q;              // [L][T][Hq][D], not rotated
    const void *cache_k;
    float *weights;             // the cache's blocks, one float a row
    int32_t req0, n_reqs;       // this launch's requests of the table (CUDA cores: all)
    int32_t n_layers, n_q_heads, n_kv_heads;
    int32_t total_q;
    int32_t max_rows;           // largest P_b + Lq_b of the launch's requests
    int32_t max_q_len;          // and longest query
    float scale_log2;
    int32_t interleaved;
    int32_t accumulate;
    int *err;
};

// ---- eviction of a cache's lightest rows ----
// Per-request data (64 bytes).
struct alignas(16) DevEvict {
    int64_t src_row0;    // cache_offsets[b] * L * H_kv
    int64_t dst_row0;    // dst_offsets[b] * L * H_kv
    int64_t kept0;       // first entry of the request's kept rows
    int32_t src_cap, dst_cap;
    int32_t n, keep;     // rows held, rows to keep (keep <= n)
    int32_t chunk0;      // first (unit, row chunk) of the request (move kernel)
    int32_t pad_[5];
};
static_assert(sizeof(DevEvict) == 64, "eviction table layout");
struct EvictTable {
    DevEvict reqs[kInlineEntries];
};
struct EvictArgs {
    const DevEvict *reqs;       // NULL: the EvictTable parameter
    const float2 *rope;
    const float2 *rope_turns;   // w_i / 2 pi in two words
    const float *weights;
    const void *cache_k, *cache_v;
    void *dst_k, *dst_v;
    float *dst_weights;         // or NULL
    int32_t *kept;
    int32_t n_reqs, units;      // units: L * H_kv
    int32_t n_first, n_recent;
    int32_t max_n;              // largest n of the batch
    int32_t max_keep;           // most rows kept of a request
    int32_t n_chunks;           // (unit, row chunk) pieces of the batch (move kernel)
    int32_t interleaved;
    int32_t keep_rotation;      // keys are copied as they are
    int32_t in_place;
};

// ---- paged cache ----
// Rows that are packed together, dims that share a scale, and the bytes of the
// keys (or values) of 16 of these rows, of both, and of a packed block.
constexpr int kPackRows = 32, kPackGroup = 32;
constexpr int kPackPart = 16 * 128 / 2 + 16 * (128 / kPackGroup) * 2;
constexpr int kPackStep = 2 * kPackPart, kPackBytes = kPackRows / 16 * kPackStep;
static_assert(kPackBytes == 4608, "packed block layout");

// Per-request data (64 bytes).  Page g of a request is entry g + off[0] of the
// call's list of page numbers where g < few, else entry g + off[1] (a window's
// list leaves out the pages between the first rows and the window).
struct alignas(16) DevPageReq {
    int32_t q_off, q_len;   // query (append: new) tokens; pack and unpack: blocks, numbered through the call
    int32_t pos0;           // position of the first token; pack and unpack: first row
    int32_t kv_len;         // rows that a query may see
    int32_t packed_len;     // rows of them that are read from the packed pages
    int32_t few, off[2];    // pages
    int32_t pfew, poff[2];  // packed pages
    int32_t item0;          // first work item of a unit (tensor-core kernel)
    int32_t tile0;          // first tile of a unit's restored rows (tensor-core kernel)
    int32_t pad_[3];
};
static_assert(sizeof(DevPageReq) == 64, "paged request table layout");
constexpr int kInlinePages = 1024;
struct PageTable {
    DevPageReq reqs[kInlineEntries];
    int32_t ids[kInlinePages];
};
// Where the rows are: row r of page i, (layer l, kv-head h), at element
// i * s_page + l * s_layer + h * s_head + r * D.
struct PageGeo {
    void *k, *v;
    int64_t s_page, s_layer, s_head;
    int32_t rows;           // rows of a page
    int32_t shift;          // their logarithm to base 2, or -1: no power of two
    uint8_t *packed;        // or NULL: packed pages, block by block
    int64_t packed_page;    // bytes of a packed page
};
struct PageArgs {
    const DevPageReq *reqs;     // NULL: the PageTable parameter holds requests and page numbers
    const int32_t *ids;
    int32_t n_reqs;
    int32_t n_layers, n_q_heads, n_kv_heads;
    int32_t total_q;            // T
    int32_t interleaved;
    const float2 *rope;
    PageGeo g;
    // attention
    const void *q;
    void *out;
    float scale_log2;
    int32_t window, n_first;    // window 0: everything before the query
    int *err;
    // append
    const void *k, *v;          // new keys and values
    int64_t s_layer, s_tok, s_head;
    int32_t turned;             // keys are at their positions already
    int32_t per_cta;            // (layer, kv-head) units of a CTA
};

// The tensor-core kernel of the paged attention: one (unit, request, 256-row block
// of its query rows, stretch of its key tiles) an item.  Packed rows are restored to
// bf16 first, by k_page_restore, in tiles of 128 rows: [unit of the slice][tile][128][D].
constexpr int64_t kPagePartBytes = 256 * 128 * 4 + 256 * 8, kPageTileBytes = 128 * 128 * 2;
struct PageTcArgs {
    int64_t total;          // items
    int32_t unit_items;     // of one (layer, kv-head)
    int32_t splits;         // stretches of a block
    int32_t box;            // rows of a TMA box of the pages; 0: no tile is loaded by TMA
    float *part;            // splits > 1: total partial results
    int32_t lh_base;        // first (layer, kv-head) unit of this launch's slice
    int32_t unit_tiles;     // restored tiles of a unit
    int32_t one_tile;       // no request has more than 128 of the kernel's rows
    int32_t out32;          // `out` is 32-byte aligned
    void *rest_k, *rest_v;  // restored rows
    const void *q_rot;      // the turned queries
};

// ---- launchers (each returns the cudaGetLastError of its launch) ----
cudaError_t launch_rope_tables(float2 *tab, int head_dim, double theta, cudaStream_t s);
// `inl` (optional) carries the span and local tables; a.spans / a.locals are
// then ignored.
cudaError_t launch_assemble(const AssembleArgs &a, int dtype, int head_dim, int n_spans,
                            cudaStream_t s, const AssembleTables *inl = nullptr);
cudaError_t launch_attention_simt(const AttnArgs &a, const ReqTable &rt, int dtype, int head_dim,
                                  cudaStream_t s);

// Tensor-core attention (bf16, head_dim 128).  `tmaps` points to two
// CUtensorMap objects (K then V) describing the cache as a 2-D
// [rows, head_dim] bf16 tensor.
// The tensor-core attention's values-gathering variant (kvr_prefill): V tiles
// of prefix rows are gathered from the pool, seen as a 2-D
// [entries * L * H_kv * entry_len, D] tensor, through the batch's span table.
struct SpanTable {
    DevSpan spans[kInlineEntries];
};
struct GatherArgs {
    const DevSpan *spans;       // the batch's spans in global memory, or NULL: the SpanTable parameter
    const DevLocal *locals;     // the batch's request-local sources in global memory; NULL in calls with none
    int32_t n_spans;            // non-empty spans of the batch (request b's start at DevReq::span0)
    int32_t entry_len;          // pool tokens per entry
    const void *pool_v;         // the pool's values (bf16)
    int64_t ps_entry, ps_layer, ps_head, ps_tok;   // their strides, in elements
    int32_t tma_pool;           // the TMA maps of the pool's values are set (a contiguous pool)
};

struct TcAttnArgs {
    AttnArgs base;
    const ReqTable *rt;         // used when base.reqs is NULL
    const void *tmap_q;         // host CUtensorMaps, passed by value to the kernel:
    const void *tmap_k;         //   rotated packed Q [L*Hkv*T*G, D], cache K and V [rows, D]
    const void *tmap_v;
    int32_t n_m_blocks;         // total 256-row query blocks over all requests
    int32_t n_sms;              // persistent grid size bound
    bool gather_v;              // V tiles of prefix rows from the pool (g, st), K from the cache
    const void *tmap_pv;        // the pool's values as [rows, D] with a one-row box (gather4)
    const void *tmap_bv;        // the same with a 32-row box (runs of consecutive pool rows)
    GatherArgs g;
    const SpanTable *st;
    const void *tmap_out;       // out as [L*T][H_q][D] with a (64, G, 32 / G) box (base.out_tma)
};
// `pdl`: the kernel before it on the stream is the assemble kernel of the
// same prefill (which it may overlap: it reads only the caller's inputs and
// writes only query-side rows).
cudaError_t launch_query_prologue(const QueryPrologueArgs &a, const ReqTable &rt, int n_sms, bool pdl,
                                  cudaStream_t s);
// `pdl`: the kernel before it on the stream is the query prologue of the
// same call; the setup (barriers, TMEM) overlaps that kernel's tail.
// Launched in two-CTA clusters when a.base.n_full < units.
cudaError_t launch_attention_tc(const TcAttnArgs &a, bool pdl, cudaStream_t s);
bool attention_tc_supported(int dtype, int head_dim);
// A decode step (every request has one query token, or none): one CTA per
// (request, layer, kv-head) rotates the step's key and query heads, appends
// the key and value at row P_b and streams the cache block (the cache tensor
// maps of the prefill attention).  Replaces the query prologue for the step.
struct DecodeIO {
    const void *kq;             // [L][T][Hkv][D], not rotated
    const void *vq;
    void *cache_k;
    void *cache_v;
    int32_t interleaved;        // RoPE pairs (x_2i, x_2i+1)
};
bool decode_supported(int dtype, int head_dim, int group);
// One CTA whose only wait (bounded by limit_ns) is on a barrier nothing
// completes: records kDevTimeout in *err when the limit runs out.
cudaError_t launch_wait_selftest(int *err, unsigned long long limit_ns, cudaStream_t s);
// `pdl`: programmatic launch (the kernel sets up while the kernel before it
// finishes, and reads nothing before that kernel is done); a decode step lets
// the next one launch that way
cudaError_t launch_decode_attention(const AttnArgs &a, const ReqTable &rt, const void *tmap_k, const void *tmap_v,
                                    const DecodeIO &io, bool pdl, cudaStream_t s);
cudaError_t launch_shared_simt(const SharedArgs &a, const SharedTable &rt, int dtype, int head_dim, int n_sms, cudaStream_t s);
// bf16, head_dim 128: rotation and append, then the prefix part and the own part
// of a slice of the units.
cudaError_t launch_shared_prologue(const SharedArgs &a, const SharedTable &rt, void *q_rot, bool pdl, cudaStream_t s);
cudaError_t launch_shared_tc(const SharedTcArgs &t, bool pdl, cudaStream_t s);
cudaError_t launch_weights_simt(const WeightsArgs &a, const ReqTable &rt, int dtype, int head_dim, int n_sms, cudaStream_t s);
// bf16, head_dim 128: the tensor-core kernel; `tmap_k` points to the CUtensorMap
// of the cache's keys ([rows, head_dim], 64 x 128 boxes).
cudaError_t launch_weights_tc(const WeightsArgs &a, const ReqTable &rt, const void *tmap_k, int n_sms, cudaStream_t s);
// Rows of one piece of the eviction's move kernel.
constexpr int kEvictChunk = 64;
cudaError_t launch_rope_turns(float2 *turns, int head_dim, double theta, cudaStream_t s);
cudaError_t launch_evict(const EvictArgs &a, const EvictTable &rt, int dtype, int head_dim, int n_sms, cudaStream_t s);
// Paged cache: rotation and append; attention; rows packed, and packed rows
// restored (bf16, head_dim 128; `n_blocks` of kPackRows rows in all).
cudaError_t launch_page_append(const PageArgs &a, const PageTable &t, int dtype, int head_dim, int n_sms, cudaStream_t s);
cudaError_t launch_page_simt(const PageArgs &a, const PageTable &t, int dtype, int head_dim, cudaStream_t s);
// Query rows (tokens times query heads of a kv head) of a request up to which k_page_decode
// takes it; `host_reqs` is the host's copy of the request table.
constexpr int kPageFewRows = 16;
// Parts of at most as many rows that a request which sees packed rows is taken in.
constexpr int kPagePackedParts = 3;
cudaError_t launch_page_decode(const PageArgs &a, const PageTable &t, const DevPageReq *host_reqs, int n_sms, cudaStream_t s);
cudaError_t launch_page_queries(const PageArgs &a, const PageTable &t, void *q_rot, cudaStream_t s);
// One slice of lh_count units: restore (unit_tiles > 0), attention, join (splits > 1).
// Host CUtensorMaps: packed queries and restored rows with 64 x 128 boxes, pages with
// 64 x box ones.
struct PageTcMaps {
    const void *q, *k, *v, *rest_k, *rest_v;
};
cudaError_t launch_page_tc(const PageArgs &a, const PageTcArgs &p, const PageTable &t, const PageTcMaps &m, int lh_count, int n_sms,
                           cudaStream_t s);
cudaError_t launch_page_pack(const PageArgs &a, const PageTable &t, int64_t n_blocks, bool unpack, cudaStream_t s);
// Whether `n_sms` CTAs of the attention kernel (either variant) can be
// resident at once as two-CTA clusters.
bool attention_tc_pairs_fit(int n_sms);

}  // namespace kvr
