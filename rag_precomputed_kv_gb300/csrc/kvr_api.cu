// kvr_api.cu -- the C ABI: validation, span tables, staging and launches.
//
// Host work per call is bookkeeping only: validate every span against its
// source and every request against its cache block, lay the span / request
// tables out (the stitched row of span i is the prefix sum of the lengths
// before it -- CoinRAG blog section 2.3), copy them to the device with one
// asynchronous H2D copy from a pinned staging slot, and launch the kernels on
// the caller's stream.  Allocations and host waits happen only where the
// header lists them: binding the pool to a device, growing a staging slot or
// the query scratch past its size (kvr_pool_reserve sizes both up front), and
// reusing a staging slot that an earlier call's work still holds.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <exception>
#include <string>
#include <vector>

#include "kvr_internal.cuh"
#include "kvr_page_common.cuh"

using namespace kvr;

namespace {

// One-line reason of the last failure on this thread (a fixed buffer: the
// error paths allocate nothing, the allocation-free entry point included).
thread_local char g_last_error[512];

kvr_status fail(kvr_status st, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_last_error, sizeof g_last_error, fmt, ap);
    va_end(ap);
    return st;
}

kvr_status cuda_fail(cudaError_t e, const char *what)
{
    return fail(KVR_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

}  // namespace

kvr_status kvr::record_error(kvr_status st, const char *msg)
{
    snprintf(g_last_error, sizeof g_last_error, "%s", msg ? msg : "");
    return st;
}

namespace {

// Staging slots per pool: a call whose tables do not fit its kernels'
// parameters takes the next slot in turn, and waits on the host only if that
// slot's previous call has not yet run (kSlots such calls queued ahead).
constexpr int kSlots = 8;

// Host-pool prefill pipeline: layer groups, and the CTAs its stitch keeps
// (the attention runs on the other SMs meanwhile).
constexpr int kMaxLayerParts = 8;
constexpr int kHostStitchCtas = 64;

// Scoped NVTX range (a profiler's timeline shows which library call and which
// kernel each stretch of host time enqueued; nothing without a profiler).
struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
};

struct Slot {
    void *host = nullptr;   // pinned: tables built by the host
    void *dev = nullptr;    // device: the uploaded tables, then per-call device scratch
    size_t host_cap = 0, dev_cap = 0;
    cudaEvent_t done = nullptr;
    bool used = false;
};

// Restores the caller's current device on scope exit.
struct DeviceGuard {
    int prev = -1;
    explicit DeviceGuard(int dev)
    {
        if (cudaGetDevice(&prev) == cudaSuccess && prev != dev)
            cudaSetDevice(dev);
        else
            prev = -1;
    }
    ~DeviceGuard()
    {
        if (prev >= 0)
            cudaSetDevice(prev);
    }
};

size_t align16(size_t x) { return (x + 15) & ~size_t(15); }

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

struct kvr_pool {
    kvr_pool_desc d{};
    int device = 0;
    int cc = 0;               // compute capability, major * 10 + minor
    float2 *rope = nullptr;   // RoPE tables, then the pairs' frequencies in turns
    float2 *rope_turns = nullptr;
    int *err = nullptr;       // device error word, then the shared-prefix calls' relay words
    uint32_t shared_calls = 0;   // shared-prefix calls on the tensor cores so far
    int32_t shared_path = KVR_SHARED_NONE;   // kernels of the last shared-prefix call
    int32_t page_path = KVR_PAGE_NONE;       // ... of the last paged attention
    Slot slots[kSlots];
    int next = 0;
    PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    bool ready = false;       // device-side setup done
    int n_sms = 1;
    // rotated, packed query heads for the tensor-core attention (grown on
    // demand); q_rot_done orders its reuse after the last call's attention
    void *q_rot = nullptr;
    size_t q_rot_cap = 0;
    cudaEvent_t q_rot_done = nullptr;
    bool q_rot_used = false;
    // partial results of the shared-prefix attention (grown on demand; used
    // and reused with the query scratch)
    void *part = nullptr;
    size_t part_cap = 0;
    // a pool in pinned host memory: kvr_prefill stitches it by layer groups on
    // a second stream, each group's attention overlapping the next group's
    // stitch (which reads over the CPU-GPU link)
    bool host_pool = false;
    cudaStream_t side = nullptr;
    cudaEvent_t side_start = nullptr;
    cudaEvent_t part_ev[kMaxLayerParts] = {};
    cudaEvent_t timing[6] = {};  // optional kernel timing events (caller-owned)
    bool timed = false;

    void mark(int i, cudaStream_t s) const
    {
        if (timed && timing[i])
            cudaEventRecord(timing[i], s);
    }

    int elt() const { return d.dtype == KVR_DTYPE_BF16 ? 2 : 4; }
    int vec_elems() const { return 16 / elt(); }

    // A staging slot with at least `host_bytes` of pinned and `dev_bytes` of
    // device memory; waits until the slot's last upload and the kernels that
    // read it are done (only when kSlots later calls have been enqueued since
    // and that work has not run yet).  A slot smaller than asked is freed and
    // allocated again (cudaFreeHost / cudaFree synchronize the device).
    kvr_status acquire(size_t host_bytes, size_t dev_bytes, Slot **out)
    {
        Slot &s = slots[next];
        next = (next + 1) % kSlots;
        cudaError_t e;
        if (s.used && cudaEventQuery(s.done) != cudaSuccess) {
            NvtxRange r("kvr.staging_slot_wait");
            if ((e = cudaEventSynchronize(s.done)) != cudaSuccess)
                return cuda_fail(e, "staging slot wait");
        }
        kvr_status st = grow(s, host_bytes, dev_bytes);
        if (st == KVR_OK)
            *out = &s;
        return st;
    }

    // Slot `s` (idle) with at least the given capacities, and its event.
    static kvr_status grow(Slot &s, size_t host_bytes, size_t dev_bytes)
    {
        cudaError_t e;
        if (s.host_cap < host_bytes) {
            NvtxRange r("kvr.staging_alloc");
            const size_t cap = std::max<size_t>({host_bytes, 2 * s.host_cap, 65536});
            if (s.host)
                cudaFreeHost(s.host);
            s.host = nullptr;
            s.host_cap = 0;
            if ((e = cudaMallocHost(&s.host, cap)) != cudaSuccess)
                return cuda_fail(e, "staging host buffer");
            s.host_cap = cap;
        }
        if (s.dev_cap < dev_bytes) {
            NvtxRange r("kvr.staging_alloc");
            const size_t cap = std::max<size_t>({dev_bytes, 2 * s.dev_cap, 65536});
            if (s.dev)
                cudaFree(s.dev);
            s.dev = nullptr;
            s.dev_cap = 0;
            if ((e = cudaMalloc(&s.dev, cap)) != cudaSuccess)
                return cuda_fail(e, "staging device buffer");
            s.dev_cap = cap;
        }
        if (!s.done && (e = cudaEventCreateWithFlags(&s.done, cudaEventDisableTiming)) != cudaSuccess)
            return cuda_fail(e, "staging event");
        return KVR_OK;
    }

    // The partial-result scratch with at least `bytes`, likewise.
    kvr_status grow_part_scratch(size_t bytes)
    {
        if (part_cap >= bytes)
            return KVR_OK;
        NvtxRange r("kvr.part_scratch_alloc");
        cudaError_t e;
        if (q_rot_used && (e = cudaEventSynchronize(q_rot_done)) != cudaSuccess)
            return cuda_fail(e, "partial result scratch wait");
        if (part)
            cudaFree(part);
        part = nullptr;
        part_cap = 0;
        if ((e = cudaMalloc(&part, bytes)) != cudaSuccess)
            return cuda_fail(e, "partial result scratch");
        part_cap = bytes;
        return KVR_OK;
    }

    // The rotated-query scratch with at least `bytes`: a smaller one is freed
    // (after the last call's attention is done with it) and allocated again.
    kvr_status grow_query_scratch(size_t bytes)
    {
        cudaError_t e;
        if (q_rot_cap < bytes) {
            NvtxRange r("kvr.query_scratch_alloc");
            if (q_rot_used && (e = cudaEventSynchronize(q_rot_done)) != cudaSuccess)
                return cuda_fail(e, "query scratch wait");
            if (q_rot)
                cudaFree(q_rot);
            q_rot = nullptr;
            q_rot_cap = 0;
            q_rot_used = false;
            if ((e = cudaMalloc(&q_rot, bytes)) != cudaSuccess)
                return cuda_fail(e, "query scratch");
            q_rot_cap = bytes;
        }
        if (!q_rot_done && (e = cudaEventCreateWithFlags(&q_rot_done, cudaEventDisableTiming)) != cudaSuccess)
            return cuda_fail(e, "query scratch event");
        return KVR_OK;
    }
};

// ---------------------------------------------------------------------------
// registration
// ---------------------------------------------------------------------------
extern "C" kvr_status kvr_pool_register(const kvr_pool_desc *desc, kvr_pool_t *out)
{
    if (!out)
        return fail(KVR_ERR_INVALID_ARG, "out is NULL");
    *out = nullptr;
    if (!desc)
        return fail(KVR_ERR_INVALID_ARG, "desc is NULL");
    const kvr_pool_desc &d = *desc;
    if (d.dtype != KVR_DTYPE_BF16 && d.dtype != KVR_DTYPE_FP32)
        return fail(KVR_ERR_UNSUPPORTED, "dtype %d", d.dtype);
    if (d.head_dim != 64 && d.head_dim != 128)
        return fail(KVR_ERR_UNSUPPORTED, "head_dim %d (64 or 128)", d.head_dim);
    if (d.n_layers < 1 || d.n_kv_heads < 1 || d.n_q_heads < 1 || d.n_q_heads % d.n_kv_heads)
        return fail(KVR_ERR_INVALID_ARG, "layers %d, q heads %d, kv heads %d", d.n_layers,
                    d.n_q_heads, d.n_kv_heads);
    if (d.n_entries < 1 || d.entry_len < 1 || d.entry_len > kMaxPosition)
        return fail(KVR_ERR_INVALID_ARG, "n_entries %lld, entry_len %lld",
                    (long long)d.n_entries, (long long)d.entry_len);
    if (d.flags & ~(KVR_POOL_KEYS_UNROTATED | KVR_POOL_ROPE_INTERLEAVED))
        return fail(KVR_ERR_INVALID_ARG, "unknown pool flags 0x%x", (unsigned)d.flags);
    if (!d.k || !d.v)
        return fail(KVR_ERR_INVALID_ARG, "pool k / v is NULL");
    if (!aligned16(d.k) || !aligned16(d.v))
        return fail(KVR_ERR_INVALID_ARG, "pool k / v not 16-byte aligned");
    if (!(d.rope_theta > 1.0) || !std::isfinite(d.rope_theta))
        return fail(KVR_ERR_INVALID_ARG, "rope_theta %g", d.rope_theta);
    const int vec = 16 / (d.dtype == KVR_DTYPE_BF16 ? 2 : 4);
    for (int i = 0; i < 4; ++i)
        if (d.stride[i] < 0 || d.stride[i] % vec)
            return fail(KVR_ERR_INVALID_ARG, "stride[%d] = %lld must be >= 0 and a multiple of %d",
                        i, (long long)d.stride[i], vec);

    kvr_pool *p = new kvr_pool();
    p->d = d;
    *out = p;
    return KVR_OK;
}

// Device-side setup, done by the first call that launches work: the RoPE
// tables for (rope_theta, head_dim), the error word, the tensor-map encoder.
static kvr_status ensure_device(kvr_pool *p)
{
    if (p->ready)
        return KVR_OK;
    cudaError_t e;
    if ((e = cudaGetDevice(&p->device)) != cudaSuccess)
        return cuda_fail(e, "cudaGetDevice");
    int maj = 0, min = 0;
    cudaDeviceGetAttribute(&maj, cudaDevAttrComputeCapabilityMajor, p->device);
    cudaDeviceGetAttribute(&min, cudaDevAttrComputeCapabilityMinor, p->device);
    p->cc = maj * 10 + min;
    cudaDeviceGetAttribute(&p->n_sms, cudaDevAttrMultiProcessorCount, p->device);
    const size_t tab = sizeof(float2) * 2 * kRopeSplit * (p->d.head_dim / 2);
    if ((e = cudaMalloc(&p->rope, tab + sizeof(float2) * (p->d.head_dim / 2))) != cudaSuccess ||
        (e = cudaMalloc(&p->err, 3 * sizeof(int))) != cudaSuccess ||
        (e = cudaMemset(p->err, 0, 3 * sizeof(int))) != cudaSuccess ||
        (e = launch_rope_tables(p->rope, p->d.head_dim, p->d.rope_theta, 0)) != cudaSuccess ||
        (e = launch_rope_turns(p->rope + 2 * kRopeSplit * (p->d.head_dim / 2), p->d.head_dim, p->d.rope_theta, 0)) !=
            cudaSuccess ||
        (e = cudaStreamSynchronize(0)) != cudaSuccess)
        return cuda_fail(e, "pool device setup");
    p->rope_turns = p->rope + 2 * kRopeSplit * (p->d.head_dim / 2);
    cudaDriverEntryPointQueryResult q;
    void *fn = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
        p->encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    cudaPointerAttributes pa{};
    if (cudaPointerGetAttributes(&pa, p->d.k) == cudaSuccess)
        p->host_pool = pa.type == cudaMemoryTypeHost;
    else
        cudaGetLastError();
    p->ready = true;
    return KVR_OK;
}

extern "C" kvr_status kvr_pool_unregister(kvr_pool_t p)
{
    if (!p)
        return KVR_OK;
    if (!p->ready) {  // device setup never completed: free what it got
        if (p->rope)
            cudaFree(p->rope);
        if (p->err)
            cudaFree(p->err);
        delete p;
        return KVR_OK;
    }
    DeviceGuard g(p->device);
    for (Slot &s : p->slots) {
        if (s.done) {
            cudaEventSynchronize(s.done);
            cudaEventDestroy(s.done);
        }
        if (s.host)
            cudaFreeHost(s.host);
        if (s.dev)
            cudaFree(s.dev);
    }
    if (p->q_rot_done) {
        cudaEventSynchronize(p->q_rot_done);
        cudaEventDestroy(p->q_rot_done);
    }
    if (p->q_rot)
        cudaFree(p->q_rot);
    if (p->part)
        cudaFree(p->part);
    if (p->side) {
        cudaStreamSynchronize(p->side);
        cudaStreamDestroy(p->side);
    }
    if (p->side_start)
        cudaEventDestroy(p->side_start);
    for (cudaEvent_t e : p->part_ev)
        if (e)
            cudaEventDestroy(e);
    if (p->rope)
        cudaFree(p->rope);
    if (p->err)
        cudaFree(p->err);
    delete p;
    return KVR_OK;
}

// The tcgen05 kernel runs for bf16 pools with head_dim 128 on sm_103.
static bool use_tensor_cores(const kvr_pool &p);

extern "C" kvr_status kvr_pool_reserve(kvr_pool_t p, int32_t max_batch, int32_t max_spans, int32_t max_locals,
                                       int64_t max_query_tokens)
{
    if (!p)
        return fail(KVR_ERR_INVALID_ARG, "pool is NULL");
    if (max_batch < 0 || max_spans < 0 || max_locals < 0 || max_query_tokens < 0 ||
        max_query_tokens > INT32_MAX)
        return fail(KVR_ERR_INVALID_ARG, "negative or too large reservation (batch %d, spans %d, locals %d, "
                    "query tokens %lld)", max_batch, max_spans, max_locals, (long long)max_query_tokens);
    NvtxRange call("kvr_pool_reserve");
    kvr_status st;
    if ((st = ensure_device(p)) != KVR_OK)
        return st;
    DeviceGuard g(p->device);
    // the largest table a call within the limits uploads: an assemble's spans
    // and local sources, or a request table with what goes beside it: append
    // spans (CUDA-core attention), groups (shared prefixes: as many as requests)
    constexpr size_t req = std::max({sizeof(DevReq), sizeof(DevShared), sizeof(DevEvict)});
    const size_t asm_bytes = align16((size_t)max_spans * sizeof(DevSpan)) + (size_t)max_locals * sizeof(DevLocal);
    const size_t append_bytes = align16((size_t)max_batch * sizeof(DevSpan)) + (size_t)max_batch * sizeof(DevLocal);
    const size_t req_bytes = align16((size_t)max_batch * req) + std::max(append_bytes, (size_t)max_batch * sizeof(DevGroup));
    const size_t page_bytes = align16((size_t)max_batch * kPagePackedParts * sizeof(DevPageReq)) + (size_t)max_spans * sizeof(int32_t);
    const size_t bytes = std::max({asm_bytes, req_bytes, page_bytes});
    cudaError_t e;
    for (Slot &s : p->slots) {
        if (s.used && (e = cudaEventSynchronize(s.done)) != cudaSuccess)
            return cuda_fail(e, "staging slot wait");
        if ((st = kvr_pool::grow(s, bytes, bytes)) != KVR_OK)
            return st;
    }
    if (use_tensor_cores(*p)) {
        const size_t q_bytes = (size_t)p->d.n_layers * (size_t)max_query_tokens * p->d.n_q_heads * p->d.head_dim * 2;
        if (q_bytes > 0 && (st = p->grow_query_scratch(q_bytes)) != KVR_OK)
            return st;
    }
    return KVR_OK;
}

static bool use_tensor_cores(const kvr_pool &p)
{
    return attention_tc_supported(p.d.dtype, p.d.head_dim) && p.cc == 103 && p.encode;
}

// ---------------------------------------------------------------------------
// assemble
// ---------------------------------------------------------------------------
namespace {

kvr_status check_offsets32(const int32_t *o, int32_t batch, const char *name)
{
    if (!o)
        return fail(KVR_ERR_INVALID_ARG, "%s is NULL", name);
    if (o[0] != 0)
        return fail(KVR_ERR_INVALID_ARG, "%s[0] = %d, must be 0", name, o[0]);
    for (int b = 0; b < batch; ++b)
        if (o[b + 1] < o[b])
            return fail(KVR_ERR_INVALID_ARG, "%s decreases at %d", name, b);
    return KVR_OK;
}

kvr_status check_cache_offsets(const int64_t *o, int32_t batch)
{
    if (!o)
        return fail(KVR_ERR_INVALID_ARG, "cache_offsets is NULL");
    if (o[0] < 0)
        return fail(KVR_ERR_INVALID_ARG, "cache_offsets[0] < 0");
    for (int b = 0; b < batch; ++b)
        if (o[b + 1] < o[b] || o[b + 1] - o[b] > kMaxPosition)
            return fail(KVR_ERR_INVALID_ARG, "cache_offsets[%d..%d] invalid", b, b + 1);
    return KVR_OK;
}

kvr_status check_local(const kvr_pool &p, const kvr_local_src &lc, int i)
{
    if (!lc.k || !lc.v || !aligned16(lc.k) || !aligned16(lc.v))
        return fail(KVR_ERR_INVALID_ARG, "local source %d: k / v NULL or not 16-byte aligned", i);
    if (lc.len < 0 || lc.len > kMaxPosition)
        return fail(KVR_ERR_INVALID_ARG, "local source %d: len %lld", i, (long long)lc.len);
    for (int s = 0; s < 3; ++s)
        if (lc.stride[s] < 0 || lc.stride[s] % p.vec_elems())
            return fail(KVR_ERR_INVALID_ARG, "local source %d: stride[%d] = %lld", i, s,
                        (long long)lc.stride[s]);
    return KVR_OK;
}

// Units of (layer, kv-head) per assemble CTA: about 256 rows per CTA.
int units_per_cta(int LH, int64_t rows, int64_t n_spans)
{
    const int64_t avg = std::max<int64_t>(1, rows / std::max<int64_t>(1, n_spans));
    return (int)std::min<int64_t>(LH, std::max<int64_t>(1, 256 / avg));
}

}  // namespace

// One assemble call, validated (host tables built), then staged (device
// tables in kernel parameters or uploaded), then launched.
struct AsmPlan {
    std::vector<DevSpan> ds;
    std::vector<int32_t> plen;
    std::vector<int32_t> span0;   // request b's first entry of ds
    int64_t flat = 0;
    const kvr_local_src *locals = nullptr;
    int32_t n_locals = 0;
    void *cache_k = nullptr, *cache_v = nullptr;
    int32_t *pos_ids = nullptr, *src_map = nullptr;
    AssembleArgs a{};
    bool inl = false;
    bool upload = false;   // upload the tables even for a small call (a later kernel reads them)
    AssembleTables tab;
    Slot *slot = nullptr;
};

static kvr_status asm_validate(const kvr_pool &p, int32_t batch, const int32_t *span_offsets,
                               const kvr_span *spans, const kvr_local_src *locals, int32_t n_locals,
                               const int64_t *cache_offsets, uint32_t flags, AsmPlan &pl)
{
    if (flags & ~(uint32_t)KVR_POSITIONS_COMPOSITE)
        return fail(KVR_ERR_INVALID_ARG, "unknown flags 0x%x", flags);
    kvr_status st;
    if ((st = check_offsets32(span_offsets, batch, "span_offsets")) != KVR_OK ||
        (st = check_cache_offsets(cache_offsets, batch)) != KVR_OK)
        return st;
    const int32_t n_spans = span_offsets[batch];
    if (n_spans > 0 && !spans)
        return fail(KVR_ERR_INVALID_ARG, "spans is NULL");
    if (n_locals < 0 || (n_locals > 0 && !locals))
        return fail(KVR_ERR_INVALID_ARG, "locals NULL with n_locals %d", n_locals);
    for (int i = 0; i < n_locals; ++i)
        if ((st = check_local(p, locals[i], i)) != KVR_OK)
            return st;
    const bool composite = flags & KVR_POSITIONS_COMPOSITE;
    const int LH = p.d.n_layers * p.d.n_kv_heads;

    pl.locals = locals;
    pl.n_locals = n_locals;
    pl.ds.reserve(n_spans);
    pl.plen.assign(batch, 0);
    pl.span0.assign(batch, 0);
    int64_t flat = 0;
    for (int b = 0; b < batch; ++b) {
        const int64_t cap = cache_offsets[b + 1] - cache_offsets[b];
        int64_t row = 0;
        pl.span0[b] = (int32_t)pl.ds.size();
        for (int i = span_offsets[b]; i < span_offsets[b + 1]; ++i) {
            const kvr_span s = spans[i];
            int64_t src_len;
            if (s.src < 0)
                return fail(KVR_ERR_OUT_OF_RANGE, "span %d: negative source id %d", i, s.src);
            if (s.src & KVR_SRC_LOCAL) {
                const int idx = s.src & ~KVR_SRC_LOCAL;
                if (idx >= n_locals)
                    return fail(KVR_ERR_OUT_OF_RANGE, "span %d: local source %d of %d", i, idx,
                                n_locals);
                src_len = locals[idx].len;
            } else {
                if (s.src >= p.d.n_entries)
                    return fail(KVR_ERR_OUT_OF_RANGE, "span %d: pool entry %d of %lld", i, s.src,
                                (long long)p.d.n_entries);
                src_len = p.d.entry_len;
            }
            if (s.start < 0 || s.end < s.start || s.end > src_len)
                return fail(KVR_ERR_OUT_OF_RANGE, "span %d: [%d, %d) outside source of %lld tokens",
                            i, s.start, s.end, (long long)src_len);
            const int32_t len = s.end - s.start;
            const int64_t pos0 = composite ? s.start : row;
            if (pos0 + len > kMaxPosition)
                return fail(KVR_ERR_OUT_OF_RANGE, "span %d: positions beyond 2^24", i);
            if (len > 0) {
                DevSpan d{};
                d.dst_row0 = cache_offsets[b] * LH;
                d.flat0 = flat;
                d.src = s.src;
                d.start = s.start;
                d.len = len;
                d.row = (int32_t)row;
                d.pos0 = (int32_t)pos0;
                d.delta = (int32_t)(pos0 - s.start);
                d.cap = (int32_t)cap;
                d.dstep = 0;
                if (!(s.src & KVR_SRC_LOCAL) && (p.d.flags & KVR_POOL_KEYS_UNROTATED)) {
                    d.delta = (int32_t)pos0;   // token t turns by its position pos0 + t
                    d.dstep = 1;
                }
                pl.ds.push_back(d);
            }
            row += len;
            flat += len;
        }
        if (row > cap)
            return fail(KVR_ERR_OUT_OF_RANGE, "request %d: prefix %lld rows > cache block %lld", b,
                        (long long)row, (long long)cap);
        pl.plen[b] = (int32_t)row;
    }
    pl.flat = flat;
    return KVR_OK;
}

static kvr_status asm_check_outputs(AsmPlan &pl, void *cache_k, void *cache_v, int32_t *pos_ids,
                                    int32_t *src_map)
{
    if (!cache_k || !cache_v || !aligned16(cache_k) || !aligned16(cache_v))
        return fail(KVR_ERR_INVALID_ARG, "cache_k / cache_v NULL or not 16-byte aligned");
    pl.cache_k = cache_k;
    pl.cache_v = cache_v;
    pl.pos_ids = pos_ids;
    pl.src_map = src_map;
    return KVR_OK;
}

// Kernel arguments and tables; large tables go up by one H2D copy from a
// pinned staging slot.  Device setup must be done.
static kvr_status asm_stage(kvr_pool *p, AsmPlan &pl, cudaStream_t s)
{
    const int LH = p->d.n_layers * p->d.n_kv_heads;
    AssembleArgs &a = pl.a;
    a.rope = p->rope;
    a.pool_k = p->d.k;
    a.pool_v = p->d.v;
    a.ps_entry = p->d.stride[0];
    a.ps_layer = p->d.stride[1];
    a.ps_head = p->d.stride[2];
    a.ps_tok = p->d.stride[3];
    a.cache_k = pl.cache_k;
    a.cache_v = pl.cache_v;
    a.pos_ids = pl.pos_ids;
    a.src_map = pl.src_map;
    a.n_layers = p->d.n_layers;
    a.n_heads = p->d.n_kv_heads;
    a.upc = units_per_cta(LH, pl.flat, (int64_t)pl.ds.size());
    a.interleaved = (p->d.flags & KVR_POOL_ROPE_INTERLEAVED) ? 1 : 0;
    const int n_locals = pl.n_locals;
    const kvr_local_src *locals = pl.locals;
    pl.inl = !pl.upload && (int)pl.ds.size() <= kInlineEntries && n_locals <= kInlineEntries;
    if (pl.inl) {
        // small call: the tables travel inside the kernel parameters
        std::memcpy(pl.tab.spans, pl.ds.data(), pl.ds.size() * sizeof(DevSpan));
        for (int i = 0; i < n_locals; ++i)
            pl.tab.locals[i] = DevLocal{locals[i].k, locals[i].v, locals[i].stride[0], locals[i].stride[1],
                                        locals[i].stride[2], locals[i].len};
        return KVR_OK;
    }
    const size_t off_loc = align16(pl.ds.size() * sizeof(DevSpan));
    const size_t bytes = off_loc + sizeof(DevLocal) * std::max(n_locals, 0);
    kvr_status st;
    if ((st = p->acquire(bytes, bytes, &pl.slot)) != KVR_OK)
        return st;
    char *h = static_cast<char *>(pl.slot->host);
    std::memcpy(h, pl.ds.data(), pl.ds.size() * sizeof(DevSpan));
    for (int i = 0; i < n_locals; ++i) {
        DevLocal l{locals[i].k, locals[i].v, locals[i].stride[0], locals[i].stride[1],
                   locals[i].stride[2], locals[i].len};
        std::memcpy(h + off_loc + i * sizeof(DevLocal), &l, sizeof l);
    }
    cudaError_t e = cudaMemcpyAsync(pl.slot->dev, h, bytes, cudaMemcpyHostToDevice, s);
    cudaEventRecord(pl.slot->done, s);   // the slot is busy from here on
    pl.slot->used = true;
    if (e != cudaSuccess)
        return cuda_fail(e, "span table upload");
    a.spans = static_cast<const DevSpan *>(pl.slot->dev);
    a.locals = reinterpret_cast<const DevLocal *>(static_cast<char *>(pl.slot->dev) + off_loc);
    return KVR_OK;
}

// `record_slot` false: the caller records the staging slot's event after the
// kernels that follow (nothing may sit between this kernel and a dependent
// launched programmatically after it).
static kvr_status asm_launch(kvr_pool *p, AsmPlan &pl, cudaStream_t s, bool record_slot = true)
{
    NvtxRange r("kvr.k_assemble");
    p->mark(0, s);
    cudaError_t e = launch_assemble(pl.a, p->d.dtype, p->d.head_dim, (int)pl.ds.size(), s,
                                    pl.inl ? &pl.tab : nullptr);
    p->mark(1, s);
    if (pl.slot && record_slot)
        cudaEventRecord(pl.slot->done, s);
    if (e != cudaSuccess)
        return cuda_fail(e, "assemble launch");
    return KVR_OK;
}

extern "C" kvr_status kvr_assemble(kvr_pool_t p, int32_t batch, const int32_t *span_offsets,
                                   const kvr_span *spans, const kvr_local_src *locals,
                                   int32_t n_locals, const int64_t *cache_offsets, void *cache_k,
                                   void *cache_v, int32_t *pos_ids, int32_t *src_map,
                                   int32_t *prefix_len, uint32_t flags, void *stream)
{
    if (!p)
        return fail(KVR_ERR_INVALID_ARG, "pool is NULL");
    if (batch < 0)
        return fail(KVR_ERR_INVALID_ARG, "batch %d", batch);
    if (batch == 0)
        return KVR_OK;
    NvtxRange call("kvr_assemble");
    AsmPlan pl;
    kvr_status st;
    if ((st = asm_validate(*p, batch, span_offsets, spans, locals, n_locals, cache_offsets, flags,
                           pl)) != KVR_OK)
        return st;
    if (prefix_len)
        std::copy(pl.plen.begin(), pl.plen.end(), prefix_len);
    if (pl.ds.empty())
        return KVR_OK;
    if ((st = asm_check_outputs(pl, cache_k, cache_v, pos_ids, src_map)) != KVR_OK ||
        (st = ensure_device(p)) != KVR_OK)
        return st;
    DeviceGuard g(p->device);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if ((st = asm_stage(p, pl, s)) != KVR_OK)
        return st;
    return asm_launch(p, pl, s);
}

// ---------------------------------------------------------------------------
// query attention
// ---------------------------------------------------------------------------
namespace {

kvr_status encode_cache_map(const kvr_pool &p, void *base, int64_t rows, CUtensorMap *m)
{
    if (!p.encode)
        return fail(KVR_ERR_UNSUPPORTED, "cuTensorMapEncodeTiled not available");
    const cuuint64_t dims[2] = {(cuuint64_t)p.d.head_dim, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)p.d.head_dim * 2};
    const cuuint32_t box[2] = {64, 128};
    const cuuint32_t estr[2] = {1, 1};
    CUresult r = p.encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(KVR_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
    return KVR_OK;
}

// The output [L * T][H_q][D] as a 3-D tensor with a box of one 64-column half
// of G heads x 32 / G tokens (a warp's 32 packed rows), 128-byte swizzle.
kvr_status encode_out_map(const kvr_pool &p, void *base, int64_t tokens, CUtensorMap *m)
{
    if (!p.encode)
        return fail(KVR_ERR_UNSUPPORTED, "cuTensorMapEncodeTiled not available");
    const int G = p.d.n_q_heads / p.d.n_kv_heads;
    const cuuint64_t dims[3] = {(cuuint64_t)p.d.head_dim, (cuuint64_t)p.d.n_q_heads, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)p.d.head_dim * 2, (cuuint64_t)p.d.n_q_heads * p.d.head_dim * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)(32 / G)};
    const cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = p.encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(KVR_ERR_CUDA, "cuTensorMapEncodeTiled (output) failed (%d)", (int)r);
    return KVR_OK;
}

// The pool as a 2-D [entries * L * H_kv * entry_len, D] tensor with a box of
// `box_rows` rows (64 columns): the values-gathering attention's TMA source.
kvr_status encode_gather_map(const kvr_pool &p, const void *base, CUtensorMap *m, uint32_t box_rows)
{
    if (!p.encode)
        return fail(KVR_ERR_UNSUPPORTED, "cuTensorMapEncodeTiled not available");
    const int64_t rows = p.d.n_entries * p.d.n_layers * p.d.n_kv_heads * p.d.entry_len;
    const cuuint64_t dims[2] = {(cuuint64_t)p.d.head_dim, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)p.d.head_dim * 2};
    const cuuint32_t box[2] = {64, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    CUresult r = p.encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box,
                          estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(KVR_ERR_CUDA, "cuTensorMapEncodeTiled (pool values) failed (%d)", (int)r);
    return KVR_OK;
}

// [rows, D] at `base` with a box of 64 columns x `box_rows` rows.
kvr_status encode_rows_map(const kvr_pool &p, const void *base, int64_t rows, uint32_t box_rows, CUtensorMap *m)
{
    if (!p.encode)
        return fail(KVR_ERR_UNSUPPORTED, "cuTensorMapEncodeTiled not available");
    const cuuint64_t dims[2] = {(cuuint64_t)p.d.head_dim, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)p.d.head_dim * 2};
    const cuuint32_t box[2] = {64, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    CUresult r = p.encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(KVR_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
    return KVR_OK;
}

// What the values-gathering attention needs beyond a query-attention launch:
// the pool's values (as a pointer, and as gather4 / 32-row box TMA sources)
// and the span table.
struct GatherLaunch {
    CUtensorMap mpv{}, mbv{};
    GatherArgs g{};
    SpanTable st;
    bool inl = false;
};

}  // namespace

// One query-attention call, validated, staged, launched (as the assemble).
struct QaPlan {
    int32_t batch = 0, T = 0, m_blocks = 0, max_lq = 0;
    const int64_t *cache_offsets = nullptr;
    const int32_t *q_offsets = nullptr;
    const void *q = nullptr, *kq = nullptr, *vq = nullptr;
    void *cache_k = nullptr, *cache_v = nullptr, *out = nullptr;
    float scale = 0.f;
    std::vector<DevReq> rq;
    std::vector<DevSpan> ap;     // the query keys / values as append spans (CUDA-core path)
    std::vector<DevLocal> al;
    bool tc = false, inl = false;
    int32_t parts = 1;           // layer groups of a host-pool prefill (attention per group)
    CUtensorMap mq, mk, mv, mo;
    ReqTable rt_inl;
    AssembleTables tab;
    AssembleArgs a{};
    AttnArgs at{};
    Slot *slot = nullptr;
};

// Host checks and tables.  T = 0 (no query token) leaves nothing to do.
static kvr_status qa_validate(const kvr_pool &p, int32_t batch, const int64_t *cache_offsets,
                              const int32_t *prefix_len, const int32_t *q_offsets, const void *q,
                              const void *kq, const void *vq, void *cache_k, void *cache_v, void *out,
                              float softmax_scale, QaPlan &pl)
{
    kvr_status st;
    if ((st = check_cache_offsets(cache_offsets, batch)) != KVR_OK ||
        (st = check_offsets32(q_offsets, batch, "q_offsets")) != KVR_OK)
        return st;
    if (!prefix_len)
        return fail(KVR_ERR_INVALID_ARG, "prefix_len is NULL");
    if (!(softmax_scale >= 0.f) || !std::isfinite(softmax_scale))
        return fail(KVR_ERR_INVALID_ARG, "softmax_scale %g", (double)softmax_scale);
    pl.T = q_offsets[batch];
    if (pl.T == 0)
        return KVR_OK;
    const void *ptrs[] = {q, kq, vq, cache_k, cache_v, out};
    for (const void *x : ptrs)
        if (!x || !aligned16(x))
            return fail(KVR_ERR_INVALID_ARG, "q / kq / vq / cache / out NULL or not 16-byte aligned");
    for (int b = 0; b < batch; ++b) {
        const int64_t cap = cache_offsets[b + 1] - cache_offsets[b];
        const int32_t P = prefix_len[b];
        const int32_t Lq = q_offsets[b + 1] - q_offsets[b];
        if (P < 0 || (int64_t)P + Lq > cap)
            return fail(KVR_ERR_OUT_OF_RANGE, "request %d: prefix %d + query %d > cache block %lld",
                        b, P, Lq, (long long)cap);
    }
    pl.batch = batch;
    pl.cache_offsets = cache_offsets;
    pl.q_offsets = q_offsets;
    pl.q = q;
    pl.kq = kq;
    pl.vq = vq;
    pl.cache_k = cache_k;
    pl.cache_v = cache_v;
    pl.out = out;
    pl.scale = softmax_scale;

    const int L = p.d.n_layers, Hkv = p.d.n_kv_heads, Hq = p.d.n_q_heads, D = p.d.head_dim;
    const int LH = L * Hkv;
    const int G = Hq / Hkv;
    const int64_t T = pl.T;
    pl.rq.resize(batch);
    for (int b = 0; b < batch; ++b) {
        const int64_t cap = cache_offsets[b + 1] - cache_offsets[b];
        const int32_t P = prefix_len[b];
        const int32_t Lq = q_offsets[b + 1] - q_offsets[b];
        pl.max_lq = std::max(pl.max_lq, Lq);
        DevReq &r = pl.rq[b];
        r.cache_row0 = cache_offsets[b] * LH;
        r.cap = (int32_t)cap;
        r.prefix = P;
        r.q_off = q_offsets[b];
        r.q_len = Lq;
        r.unit0 = 0;   // set by the schedule (tensor-core path)
        r.span0 = r.span_end = 0;
        pl.m_blocks += (int32_t)((int64_t(G) * Lq + 255) / 256);
        if (Lq > 0) {
            // the query tokens' keys / values become cache rows P..P+Lq-1;
            // their keys arrive un-rotated, so token t turns by P + t
            DevSpan d{};
            d.dst_row0 = r.cache_row0;
            d.flat0 = 0;
            d.src = KVR_SRC_LOCAL | (int32_t)pl.al.size();
            d.start = 0;
            d.len = Lq;
            d.row = P;
            d.pos0 = P;
            d.delta = P;
            d.cap = (int32_t)cap;
            d.dstep = 1;
            pl.ap.push_back(d);
            const int64_t off = (int64_t)q_offsets[b] * Hkv * D * p.elt();
            DevLocal l{static_cast<const char *>(kq) + off, static_cast<const char *>(vq) + off,
                       T * Hkv * D, D, (int64_t)Hkv * D, Lq};
            pl.al.push_back(l);
        }
    }
    return KVR_OK;
}

// Scratch, tensor maps and tables.  Device setup must be done.
static kvr_status qa_stage(kvr_pool *p, QaPlan &pl, cudaStream_t s)
{
    const int L = p->d.n_layers, Hkv = p->d.n_kv_heads, Hq = p->d.n_q_heads, D = p->d.head_dim;
    const int LH = L * Hkv;
    const int32_t batch = pl.batch, T = pl.T;
    kvr_status st;
    cudaError_t e;
    pl.tc = use_tensor_cores(*p);
    if (pl.tc) {
        // rotated packed Q scratch and the three tensor maps
        const int64_t rows = pl.cache_offsets[batch] * LH;
        const int64_t q_rows = (int64_t)L * T * Hq;
        if (rows > (int64_t)INT32_MAX - 256 || q_rows > (int64_t)INT32_MAX - 256)   // int32 TMA coordinates
            return fail(KVR_ERR_UNSUPPORTED, "cache or query rows exceed the int32 TMA coordinate range");
        if ((st = p->grow_query_scratch((size_t)q_rows * D * 2)) != KVR_OK)
            return st;
        if ((st = encode_cache_map(*p, p->q_rot, q_rows, &pl.mq)) != KVR_OK ||
            (st = encode_cache_map(*p, pl.cache_k, rows, &pl.mk)) != KVR_OK ||
            (st = encode_cache_map(*p, pl.cache_v, rows, &pl.mv)) != KVR_OK)
            return st;
        // G a power of two and `out` in device memory: the attention's epilogue
        // writes each warp's 32 rows (32 / G whole tokens) with one TMA store
        const int G = Hq / Hkv;
        pl.at.out_tma = 0;
        if ((G & (G - 1)) == 0 && G <= 32) {
            cudaPointerAttributes pa{};
            if (cudaPointerGetAttributes(&pa, pl.out) == cudaSuccess && pa.type == cudaMemoryTypeDevice) {
                if ((st = encode_out_map(*p, pl.out, (int64_t)L * T, &pl.mo)) != KVR_OK)
                    return st;
                pl.at.out_tma = 1;
            } else {
                cudaGetLastError();
            }
        }
        // the previous call's attention must be done with the query scratch
        if (p->q_rot_used && (e = cudaStreamWaitEvent(s, p->q_rot_done, 0)) != cudaSuccess)
            return cuda_fail(e, "query scratch ordering");
    }

    if (pl.tc) {
        // schedule: requests with the longest key range first (requests
        // without query tokens last), each request's units numbered after the
        // previous one's; the table goes up in this order
        std::stable_sort(pl.rq.begin(), pl.rq.end(), [](const DevReq &x, const DevReq &y) {
            if ((x.q_len > 0) != (y.q_len > 0))
                return x.q_len > 0;
            return x.prefix + x.q_len > y.prefix + y.q_len;
        });
        int64_t u0 = 0;
        for (DevReq &r : pl.rq) {
            r.unit0 = (int32_t)u0;
            u0 += ((int64_t)(Hq / Hkv) * r.q_len + 255) / 256 * (LH / pl.parts);
        }
    }

    pl.inl = batch <= kInlineEntries;   // then ap, al have <= batch entries too
    AssembleArgs &a = pl.a;
    AttnArgs &at = pl.at;
    if (pl.inl) {
        std::memcpy(pl.rt_inl.reqs, pl.rq.data(), pl.rq.size() * sizeof(DevReq));
        std::memcpy(pl.tab.spans, pl.ap.data(), pl.ap.size() * sizeof(DevSpan));
        std::memcpy(pl.tab.locals, pl.al.data(), pl.al.size() * sizeof(DevLocal));
        at.reqs = nullptr;
    } else {
        const size_t off_sp = align16(pl.rq.size() * sizeof(DevReq));
        const size_t off_lc = off_sp + align16(pl.ap.size() * sizeof(DevSpan));
        const size_t bytes = off_lc + pl.al.size() * sizeof(DevLocal);
        if ((st = p->acquire(bytes, bytes, &pl.slot)) != KVR_OK)
            return st;
        char *h = static_cast<char *>(pl.slot->host);
        char *dv = static_cast<char *>(pl.slot->dev);
        std::memcpy(h, pl.rq.data(), pl.rq.size() * sizeof(DevReq));
        std::memcpy(h + off_sp, pl.ap.data(), pl.ap.size() * sizeof(DevSpan));
        std::memcpy(h + off_lc, pl.al.data(), pl.al.size() * sizeof(DevLocal));
        e = cudaMemcpyAsync(dv, h, bytes, cudaMemcpyHostToDevice, s);
        cudaEventRecord(pl.slot->done, s);   // the slot is busy from here on
        pl.slot->used = true;
        if (e != cudaSuccess)
            return cuda_fail(e, "request table upload");
        a.spans = reinterpret_cast<const DevSpan *>(dv + off_sp);
        a.locals = reinterpret_cast<const DevLocal *>(dv + off_lc);
        at.reqs = reinterpret_cast<const DevReq *>(dv);
    }

    at.n_reqs = batch;
    at.rope = p->rope;
    at.q = pl.q;
    at.cache_k = pl.cache_k;
    at.cache_v = pl.cache_v;
    at.out = pl.out;
    at.n_layers = L;
    at.n_q_heads = Hq;
    at.n_kv_heads = Hkv;
    at.total_q = T;
    at.scale_log2 = (pl.scale > 0.f ? pl.scale : 1.f / std::sqrt((float)D)) * 1.4426950408889634f;
    at.err = p->err;
    at.interleaved = (p->d.flags & KVR_POOL_ROPE_INTERLEAVED) ? 1 : 0;
    // CUDA-core path: the query keys / values are appended by the assemble
    // kernel (un-rotated source, token t turned by P + t); the query heads
    // are rotated inside the CUDA-core attention kernel
    a.rope = p->rope;
    a.cache_k = pl.cache_k;
    a.cache_v = pl.cache_v;
    a.n_layers = L;
    a.n_heads = Hkv;
    a.upc = 1;
    a.interleaved = at.interleaved;
    return KVR_OK;
}

// `after_assemble`: the kernel just enqueued on `s` is the assemble kernel of
// the same prefill, so the query prologue may overlap it.  Without the timing
// hook the attention kernel always overlaps the prologue's tail.
static kvr_status qa_launch(kvr_pool *p, QaPlan &pl, cudaStream_t s, bool after_assemble,
                            const GatherLaunch *gl = nullptr)
{
    static const ReqTable no_reqs{};
    const ReqTable &rt = pl.inl ? pl.rt_inl : no_reqs;
    const int D = p->d.head_dim;
    cudaError_t e;
    if (pl.tc) {
        // a host-pool prefill in layer groups, stitched last group first: the
        // attention of group g runs on the SMs the stitch leaves, beside the
        // stitch of group g - 1, once the stitch of group g is done
        const int n_sms = pl.parts > 1 ? p->n_sms - kHostStitchCtas : p->n_sms;
        const int lh_part = p->d.n_layers * p->d.n_kv_heads / pl.parts;
        TcAttnArgs ta{pl.at, &rt, &pl.mq, &pl.mk, &pl.mv, pl.m_blocks, n_sms};
        ta.tmap_out = &pl.mo;
        if (pl.parts > 1)
            ta.base.lh_count = lh_part;
        // the last wave's units split in two halves of their keys when two
        // halves of each fit one wave and the grid can run as two-CTA clusters
        const int64_t units = (int64_t)pl.m_blocks * lh_part;
        const int64_t tail = units % n_sms;
        ta.base.n_full = (int32_t)units;
        if (tail > 0 && 2 * tail <= n_sms && attention_tc_pairs_fit(n_sms))
            ta.base.n_full = (int32_t)(units - tail);
        QueryPrologueArgs qp{pl.at.reqs, p->rope, pl.q, pl.kq, pl.vq, pl.cache_k, pl.cache_v, p->q_rot,
                             p->d.n_layers, p->d.n_q_heads, p->d.n_kv_heads, pl.T, pl.max_lq, pl.batch,
                             pl.at.interleaved};
        // a decode step (one query token per request): one kernel rotates,
        // appends and streams each cache block
        const bool decode = !gl && pl.max_lq == 1 &&
                            decode_supported(p->d.dtype, D, p->d.n_q_heads / p->d.n_kv_heads);
        p->mark(2, s);
        if (!decode) {
            NvtxRange r("kvr.k_query_prologue");
            e = launch_query_prologue(qp, rt, p->n_sms, after_assemble && !p->timed, s);
        } else {
            e = cudaSuccess;
        }
        p->mark(3, s);
        if (e == cudaSuccess && decode) {
            const DecodeIO io{pl.kq, pl.vq, pl.cache_k, pl.cache_v, pl.at.interleaved};
            p->mark(4, s);
            {
                NvtxRange r("kvr.k_decode_attention");
                e = launch_decode_attention(pl.at, rt, &pl.mk, &pl.mv, io, !p->timed, s);
            }
            p->mark(5, s);
        } else if (e == cudaSuccess) {
            NvtxRange r(gl ? "kvr.k_attention_tc_values_gathered" : "kvr.k_attention_tc");
            if (pl.parts > 1) {
                p->mark(4, s);
                for (int g = pl.parts - 1; g >= 0 && e == cudaSuccess; --g) {
                    if ((e = cudaStreamWaitEvent(s, p->part_ev[g], 0)) != cudaSuccess)
                        break;
                    ta.base.lh_base = g * lh_part;
                    e = launch_attention_tc(ta, false, s);
                }
                p->mark(5, s);
            } else {
                if (gl) {
                    ta.gather_v = true;
                    ta.tmap_pv = &gl->mpv;
                    ta.tmap_bv = &gl->mbv;
                    ta.g = gl->g;
                    ta.st = gl->inl ? &gl->st : nullptr;
                }
                p->mark(4, s);
                e = launch_attention_tc(ta, !p->timed, s);
                p->mark(5, s);
            }
        }
        cudaEventRecord(p->q_rot_done, s);
        p->q_rot_used = true;
    } else {
        NvtxRange r("kvr.k_attention_simt");
        p->mark(2, s);
        e = launch_assemble(pl.a, p->d.dtype, D, (int)pl.ap.size(), s, pl.inl ? &pl.tab : nullptr);
        p->mark(3, s);
        if (e == cudaSuccess) {
            p->mark(4, s);
            e = launch_attention_simt(pl.at, rt, p->d.dtype, D, s);
            p->mark(5, s);
        }
    }
    if (pl.slot)
        cudaEventRecord(pl.slot->done, s);
    if (e != cudaSuccess)
        return cuda_fail(e, "attention launch");
    return KVR_OK;
}

extern "C" kvr_status kvr_query_attention(kvr_pool_t p, int32_t batch, const int64_t *cache_offsets,
                                          const int32_t *prefix_len, const int32_t *q_offsets,
                                          const void *q, const void *kq, const void *vq,
                                          void *cache_k, void *cache_v, void *out,
                                          float softmax_scale, void *stream)
{
    if (!p)
        return fail(KVR_ERR_INVALID_ARG, "pool is NULL");
    if (batch < 0)
        return fail(KVR_ERR_INVALID_ARG, "batch %d", batch);
    if (batch == 0)
        return KVR_OK;
    NvtxRange call("kvr_query_attention");
    QaPlan pl;
    kvr_status st;
    if ((st = qa_validate(*p, batch, cache_offsets, prefix_len, q_offsets, q, kq, vq, cache_k, cache_v,
                          out, softmax_scale, pl)) != KVR_OK)
        return st;
    if (pl.T == 0)
        return KVR_OK;
    if ((st = ensure_device(p)) != KVR_OK)
        return st;
    DeviceGuard g(p->device);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if ((st = qa_stage(p, pl, s)) != KVR_OK)
        return st;
    return qa_launch(p, pl, s, false);
}

// ---------------------------------------------------------------------------
// prefill = assemble + query attention in one call
// ---------------------------------------------------------------------------
extern "C" kvr_status kvr_prefill(kvr_pool_t p, int32_t batch, const int32_t *span_offsets,
                                  const kvr_span *spans, const kvr_local_src *locals, int32_t n_locals,
                                  const int64_t *cache_offsets, void *cache_k, void *cache_v,
                                  int32_t *pos_ids, int32_t *src_map, int32_t *prefix_len,
                                  uint32_t flags, const int32_t *q_offsets, const void *q,
                                  const void *kq, const void *vq, void *out, float softmax_scale,
                                  void *stream)
{
    if (!p)
        return fail(KVR_ERR_INVALID_ARG, "pool is NULL");
    if (batch < 0)
        return fail(KVR_ERR_INVALID_ARG, "batch %d", batch);
    if (batch == 0)
        return KVR_OK;
    NvtxRange call("kvr_prefill");
    // every check of both halves before anything is enqueued
    const bool gather = flags & KVR_PREFILL_SKIP_PREFIX_CACHE;
    // the pool seen as one 2-D [rows, D] tensor for TMA box loads of value tiles
    bool tma_pool = false;
    if (gather) {
        const kvr_pool_desc &d = p->d;
        const int64_t E = d.entry_len, D = d.head_dim;
        tma_pool = d.stride[3] == D && d.stride[2] == E * D && d.stride[1] == d.n_kv_heads * E * D &&
                   d.stride[0] == (int64_t)d.n_layers * d.n_kv_heads * E * D &&
                   d.n_entries * d.n_layers * d.n_kv_heads * E <= INT32_MAX;
        if (d.dtype != KVR_DTYPE_BF16 || D != 128)
            return fail(KVR_ERR_UNSUPPORTED, "KVR_PREFILL_SKIP_PREFIX_CACHE needs a bf16 pool with head_dim 128");
    }
    AsmPlan ap;
    QaPlan qp;
    kvr_status st;
    if ((st = asm_validate(*p, batch, span_offsets, spans, locals, n_locals, cache_offsets,
                           flags & ~(uint32_t)KVR_PREFILL_SKIP_PREFIX_CACHE, ap)) != KVR_OK ||
        (st = qa_validate(*p, batch, cache_offsets, ap.plen.data(), q_offsets, q, kq, vq, cache_k,
                          cache_v, out, softmax_scale, qp)) != KVR_OK)
        return st;
    const bool stitch = !ap.ds.empty();
    if (stitch && (st = asm_check_outputs(ap, cache_k, cache_v, pos_ids, src_map)) != KVR_OK)
        return st;
    if (prefix_len)
        std::copy(ap.plen.begin(), ap.plen.end(), prefix_len);
    if (!stitch && qp.T == 0)
        return KVR_OK;
    if ((st = ensure_device(p)) != KVR_OK)
        return st;
    DeviceGuard g(p->device);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (gather) {
        // the stitch writes the prefix keys (re-rotated) and the maps only; the
        // attention reads the keys from the cache and gathers the prefix values
        // from the pool
        if (!use_tensor_cores(*p))
            return fail(KVR_ERR_UNSUPPORTED, "KVR_PREFILL_SKIP_PREFIX_CACHE needs the tensor-core attention");
        cudaPointerAttributes pa{};
        if (cudaPointerGetAttributes(&pa, p->d.k) != cudaSuccess || pa.type != cudaMemoryTypeDevice) {
            cudaGetLastError();
            return fail(KVR_ERR_UNSUPPORTED, "KVR_PREFILL_SKIP_PREFIX_CACHE needs the pool in device memory");
        }
        if (qp.T == 0)
            return KVR_OK;
        GatherLaunch gl;
        gl.g.pool_v = p->d.v;
        gl.g.ps_entry = p->d.stride[0];
        gl.g.ps_layer = p->d.stride[1];
        gl.g.ps_head = p->d.stride[2];
        gl.g.ps_tok = p->d.stride[3];
        gl.g.tma_pool = tma_pool ? 1 : 0;
        if (tma_pool && ((st = encode_gather_map(*p, p->d.v, &gl.mpv, 1)) != KVR_OK ||
                         (st = encode_gather_map(*p, p->d.v, &gl.mbv, 32)) != KVR_OK))
            return st;
        for (int b = 0; b < batch; ++b) {
            DevReq &r = qp.rq[b];
            r.span0 = ap.span0[b];
            r.span_end = b + 1 < batch ? ap.span0[b + 1] : (int32_t)ap.ds.size();
            // spans of 96 rows or more on average, all from a pool that TMA can
            // address as one tensor: the prefix value tiles go through TMA box
            // loads (runs of 32 pool rows), else through the gather warps
            const int64_t n_sp = r.span_end - r.span0;
            bool long_pool_spans = tma_pool && n_sp > 0 && (int64_t)ap.plen[b] >= 96 * n_sp;
            for (int i = r.span0; long_pool_spans && i < r.span_end; ++i)
                long_pool_spans = (ap.ds[i].src & KVR_SRC_LOCAL) == 0;
            r.flags = long_pool_spans ? kReqValuesTma : 0;
        }
        // the attention reads the local-source table from device memory
        ap.upload = n_locals > 0;
        if ((stitch && (st = asm_stage(p, ap, s)) != KVR_OK) || (st = qa_stage(p, qp, s)) != KVR_OK)
            return st;
        gl.inl = !stitch || ap.inl;
        if (stitch && ap.inl)
            std::memcpy(gl.st.spans, ap.tab.spans, ap.ds.size() * sizeof(DevSpan));
        gl.g.spans = gl.inl ? nullptr : ap.a.spans;
        // (NULL when no span names a request-local source: the attention then
        // runs its pool-only variant)
        gl.g.locals = n_locals > 0 && !gl.inl ? ap.a.locals : nullptr;
        gl.g.n_spans = (int32_t)ap.ds.size();
        gl.g.entry_len = (int32_t)p->d.entry_len;
        if (stitch) {
            ap.a.keys_only = 1;
            if ((st = asm_launch(p, ap, s, false)) != KVR_OK) {
                if (ap.slot)
                    cudaEventRecord(ap.slot->done, s);
                return st;
            }
        }
        st = qa_launch(p, qp, s, stitch, &gl);
        if (ap.slot)
            cudaEventRecord(ap.slot->done, s);
        return st;
    }
    // a pool in pinned host memory: layer groups, whose stitch (bound by the
    // CPU-GPU link, on a bounded grid and a second stream) overlaps the
    // previous group's attention
    const int L = p->d.n_layers;
    if (p->host_pool && stitch && qp.max_lq > 1 && use_tensor_cores(*p))
        for (int n = kMaxLayerParts; n > 1; --n)
            if (L % n == 0) {
                qp.parts = n;
                break;
            }
    // uploads and stream waits first, so that the kernels follow one another
    // on the stream with nothing in between
    if ((stitch && (st = asm_stage(p, ap, s)) != KVR_OK) ||
        (qp.T > 0 && (st = qa_stage(p, qp, s)) != KVR_OK))
        return st;
    if (qp.parts > 1) {
        cudaError_t e = cudaSuccess;
        if (!p->side && (e = cudaStreamCreateWithFlags(&p->side, cudaStreamNonBlocking)) != cudaSuccess)
            return cuda_fail(e, "host-pool stitch stream");
        if (!p->side_start && (e = cudaEventCreateWithFlags(&p->side_start, cudaEventDisableTiming)) != cudaSuccess)
            return cuda_fail(e, "host-pool stitch event");
        for (int g = 0; g < qp.parts; ++g)
            if (!p->part_ev[g] && (e = cudaEventCreateWithFlags(&p->part_ev[g], cudaEventDisableTiming)) != cudaSuccess)
                return cuda_fail(e, "host-pool stitch event");
        // the stitch stream starts after everything the caller's stream holds
        if ((e = cudaEventRecord(p->side_start, s)) != cudaSuccess ||
            (e = cudaStreamWaitEvent(p->side, p->side_start, 0)) != cudaSuccess)
            return cuda_fail(e, "host-pool stitch ordering");
        // The last 128-key tile of a request's last block reaches into the
        // first rows of the next request's first block, which the last stitch
        // group (the first layers) writes: until then those prefix rows' values
        // must be finite, since a masked key has weight 0 but 0 x NaN is NaN.
        const int LHn = L * p->d.n_kv_heads;
        const size_t row_bytes = (size_t)p->d.head_dim * p->elt();
        for (int b = 1; b < batch && e == cudaSuccess; ++b) {
            const int64_t rows = std::min<int64_t>(ap.plen[b], 128);
            if (rows > 0)
                e = cudaMemsetAsync(static_cast<char *>(cache_v) + (size_t)cache_offsets[b] * LHn * row_bytes, 0,
                                    (size_t)rows * row_bytes, p->side);
        }
        const int lh_part = LHn / qp.parts;
        for (int g = qp.parts - 1; g >= 0 && e == cudaSuccess; --g) {
            NvtxRange r("kvr.k_assemble_loop");
            AssembleArgs a = ap.a;
            a.lh_begin = g * lh_part;
            a.lh_count = lh_part;
            a.max_ctas = kHostStitchCtas;
            if ((e = launch_assemble(a, p->d.dtype, p->d.head_dim, (int)ap.ds.size(), p->side,
                                     ap.inl ? &ap.tab : nullptr)) == cudaSuccess)
                e = cudaEventRecord(p->part_ev[g], p->side);
        }
        if (e != cudaSuccess) {
            if (ap.slot)
                cudaEventRecord(ap.slot->done, s);
            return cuda_fail(e, "host-pool stitch launch");
        }
        st = qa_launch(p, qp, s, false);
        if (ap.slot)   // after the last group's attention, which waited for every stitch group
            cudaEventRecord(ap.slot->done, s);
        return st;
    }
    if (stitch && (st = asm_launch(p, ap, s, false)) != KVR_OK) {
        if (ap.slot)
            cudaEventRecord(ap.slot->done, s);
        return st;
    }
    if (qp.T > 0)
        st = qa_launch(p, qp, s, stitch);
    if (ap.slot)
        cudaEventRecord(ap.slot->done, s);
    return st;
}

// ---------------------------------------------------------------------------
// shared prefixes, key weights, eviction
// ---------------------------------------------------------------------------
namespace {

// One shared-prefix call: its request table, and the append of the query
// tokens' keys and values.
struct SharedPlan {
    std::vector<DevShared> rq;
    SharedTable tab;
    AssembleTables atab;
    std::vector<DevGroup> gr;   // tensor-core path
    GroupTable gtab;
};

// Partial results of the prefix part that one launch may hold; a call with
// more goes through its (layer, kv-head) units in slices.
constexpr int64_t kMaxPartBytes = int64_t(1) << 30;

// A C entry point lets no exception out (the tables are std::vectors).
template <typename F>
kvr_status guarded(F &&f)
{
    try {
        return f();
    } catch (const std::exception &e) {
        return fail(KVR_ERR_CUDA, "host allocation failed: %s", e.what());
    }
}

// A call on a stream that is being captured may only enqueue kernels: binding
// the pool, staging slots and scratch wait, allocate or are reused by later
// calls, which a replayed graph would not see.
kvr_status check_capture(const kvr_pool &p, cudaStream_t s, bool kernels_only, const char *why)
{
    cudaStreamCaptureStatus c = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(s, &c) != cudaSuccess) {
        cudaGetLastError();
        if (p.ready)   // no GPU, or a legacy stream beside a capture: the launch itself will report it
            return KVR_OK;
        c = cudaStreamCaptureStatusNone;
    }
    if (c == cudaStreamCaptureStatusNone)
        return KVR_OK;
    if (!p.ready)
        return fail(KVR_ERR_UNSUPPORTED, "the stream is being captured: bind the pool first (kvr_pool_reserve)");
    if (!kernels_only)
        return fail(KVR_ERR_UNSUPPORTED, "the stream is being captured: %s", why);
    return KVR_OK;
}

// The table `rows` on the device, through the next staging slot (whose event
// the caller records after the kernels that read it).
kvr_status upload_table(kvr_pool *p, const void *rows, size_t bytes, cudaStream_t s, Slot **slot)
{
    kvr_status st;
    if ((st = p->acquire(bytes, bytes, slot)) != KVR_OK)
        return st;
    std::memcpy((*slot)->host, rows, bytes);
    const cudaError_t e = cudaMemcpyAsync((*slot)->dev, (*slot)->host, bytes, cudaMemcpyHostToDevice, s);
    cudaEventRecord((*slot)->done, s);
    (*slot)->used = true;
    return e == cudaSuccess ? KVR_OK : cuda_fail(e, "table upload");
}

struct Range {
    const char *lo, *hi;
    bool meets(const Range &o) const { return lo < hi && o.lo < o.hi && lo < o.hi && o.lo < hi; }
};
Range range_of(const void *p, int64_t first, int64_t last, int64_t bytes)
{
    const char *c = static_cast<const char *>(p);
    return c ? Range{c + first * bytes, c + last * bytes} : Range{nullptr, nullptr};
}

// The CUDA-core path: the query tokens' keys and values become own rows
// S_b .. S_b + Lq - 1, turned by their positions P_g + S_b + t (an assemble of
// un-rotated request-local sources), then the attention.
kvr_status shared_simt(kvr_pool *p, SharedPlan &pl, SharedArgs &sa, cudaStream_t s)
{
    const int H = sa.n_kv_heads, D = p->d.head_dim;
    std::vector<DevSpan> ap;
    std::vector<DevLocal> al;
    for (const DevShared &r : pl.rq) {
        if (r.q_len == 0)
            continue;
        DevSpan d{};
        d.dst_row0 = r.cache_row0;
        d.src = KVR_SRC_LOCAL | (int32_t)al.size();
        d.len = r.q_len;
        d.row = r.own;
        d.pos0 = d.delta = r.pre_len + r.own;
        d.cap = r.cap;
        d.dstep = 1;
        ap.push_back(d);
        const int64_t off = (int64_t)r.q_off * H * D * p->elt();
        al.push_back(DevLocal{static_cast<const char *>(sa.kq) + off, static_cast<const char *>(sa.vq) + off,
                              (int64_t)sa.total_q * H * D, D, (int64_t)H * D, r.q_len});
    }
    AssembleArgs a{};
    a.rope = p->rope;
    a.cache_k = sa.cache_k;
    a.cache_v = sa.cache_v;
    a.n_layers = sa.n_layers;
    a.n_heads = H;
    a.upc = 1;
    a.interleaved = sa.interleaved;
    Slot *slot = nullptr;
    const bool inl = sa.n_reqs <= kInlineEntries;
    kvr_status st;
    if (inl) {
        std::memcpy(pl.tab.reqs, pl.rq.data(), pl.rq.size() * sizeof(DevShared));
        std::memcpy(pl.atab.spans, ap.data(), ap.size() * sizeof(DevSpan));
        std::memcpy(pl.atab.locals, al.data(), al.size() * sizeof(DevLocal));
    } else {
        const size_t off_sp = align16(pl.rq.size() * sizeof(DevShared));
        const size_t off_lc = off_sp + align16(ap.size() * sizeof(DevSpan));
        std::vector<char> rows(off_lc + al.size() * sizeof(DevLocal));
        std::memcpy(rows.data(), pl.rq.data(), pl.rq.size() * sizeof(DevShared));
        std::memcpy(rows.data() + off_sp, ap.data(), ap.size() * sizeof(DevSpan));
        std::memcpy(rows.data() + off_lc, al.data(), al.size() * sizeof(DevLocal));
        if ((st = upload_table(p, rows.data(), rows.size(), s, &slot)) != KVR_OK)
            return st;
        const char *dv = static_cast<const char *>(slot->dev);
        sa.reqs = reinterpret_cast<const DevShared *>(dv);
        a.spans = reinterpret_cast<const DevSpan *>(dv + off_sp);
        a.locals = reinterpret_cast<const DevLocal *>(dv + off_lc);
    }
    p->shared_path = KVR_SHARED_CUDA_CORES;
    p->mark(2, s);
    cudaError_t e = launch_assemble(a, p->d.dtype, D, (int)ap.size(), s, inl ? &pl.atab : nullptr);
    p->mark(3, s);
    if (e == cudaSuccess) {
        NvtxRange r("kvr.k_shared_simt");
        p->mark(4, s);
        e = launch_shared_simt(sa, pl.tab, p->d.dtype, D, p->n_sms, s);
        p->mark(5, s);
    }
    if (slot)
        cudaEventRecord(slot->done, s);
    return e == cudaSuccess ? KVR_OK : cuda_fail(e, "shared-prefix attention launch");
}

// The tensor-core path: rotation and append, then, slice by slice of the
// units, the prefix part and the own part.
kvr_status shared_tc(kvr_pool *p, SharedPlan &pl, SharedArgs &sa, int32_t n_groups, const int32_t *group_offsets,
                     const int64_t *prefix_offsets, const int32_t *prefix_len, bool any_prefix, const int32_t *q_offsets,
                     int64_t own_rows, int64_t pre_rows, cudaStream_t s)
{
    const int L = sa.n_layers, H = sa.n_kv_heads, Hq = sa.n_q_heads, D = p->d.head_dim, LH = L * H, G = Hq / H;
    SharedPrefixArgs pa{};
    sa.relay = pa.relay = reinterpret_cast<uint32_t *>(p->err + 1);
    sa.call = pa.call = ++p->shared_calls;
    pa.group = G;
    pa.total_q = sa.total_q;
    pa.scale_log2 = sa.scale_log2;
    pa.err = p->err;
    // groups with prefix and tokens first, numbered pair by pair; the others behind them
    pl.gr.reserve(n_groups);
    std::vector<int32_t> place(n_groups);
    int64_t own_tiles = 0;   // that the 256-row blocks of a unit meet
    bool all_active = true;
    for (int pass = 0; pass < 2; ++pass)
        for (int g = 0; g < n_groups; ++g) {
            const int32_t t0 = q_offsets[group_offsets[g]], t1 = q_offsets[group_offsets[g + 1]];
            const bool active = prefix_len[g] > 0 && t1 > t0;
            if (active != (pass == 0))
                continue;
            if ((int64_t)(t1 - t0) * G > INT32_MAX - 256)
                return fail(KVR_ERR_UNSUPPORTED, "group %d: too many query rows", g);
            DevGroup d{};
            d.pre_row0 = prefix_offsets[g] * LH;
            d.pre_cap = (int32_t)(prefix_offsets[g + 1] - prefix_offsets[g]);
            d.pre_len = prefix_len[g];
            d.q_off = t0;
            d.rows = (t1 - t0) * G;
            if (active) {
                d.nt = (d.pre_len + 127) / 128;
                d.mb = (d.rows + 255) / 256;
                d.item0 = pa.unit_blocks;
                d.w0 = pa.unit_pairs;
                pa.unit_blocks += d.mb;
                pa.unit_pairs += (int64_t)d.mb * d.nt;
                int b = group_offsets[g];
                for (int m = 0; m < d.mb; ++m) {
                    const int32_t first = t0 + m * 256 / G;
                    const int32_t end = t0 + (std::min(d.rows, m * 256 + 256) - 1) / G + 1;
                    while (pl.rq[b].q_off + pl.rq[b].q_len <= first)
                        ++b;
                    for (int i = b; i < group_offsets[g + 1] && pl.rq[i].q_off < end; ++i)
                        if (pl.rq[i].q_len > 0)
                            own_tiles += (pl.rq[i].own + std::min(pl.rq[i].q_len, end - pl.rq[i].q_off) + 127) / 128;
                }
            } else {
                d.item0 = pa.unit_blocks;
                d.w0 = pa.unit_pairs;
                all_active = all_active && t1 == t0;
            }
            place[g] = (int32_t)pl.gr.size();
            pl.gr.push_back(d);
        }
    // One kernel for whole blocks, their own keys and the output, where blocks are
    // well filled, meet few own tiles, and come out even over the SMs: in units of
    // a key tile (2 us for 256 rows), a round of whole blocks costs its tiles and
    // 1.7 more, and partial results with an own part cost 1.15 a tile, 6.3 a block
    // and 6 a call.  Measured on 2 x 8 requests of 64 tokens x 7 heads on 2,592
    // rows, 26 blocks a unit, n units: n = 4: 54 us against 59; 8 (1.4 blocks an
    // SM, two rounds): 101 against 96; 16: 151 against 184; 112: 928 against 1,070.
    // 8 of 70 x 4 on 400 rows, 288 units: 338 against 443.  Blocks of few rows wait
    // for each tile in turn: 8 groups of one 4-row request on 2,000 rows: 451
    // against 391.  Four own tiles a block: 292 against 222 for 16 requests of 20 x
    // 4 rows on 500.
    bool whole = false;
    if (all_active && pa.unit_blocks > 0 && sa.total_q * (int64_t)G >= 128 * pa.unit_blocks &&
        own_tiles <= 3 * pa.unit_blocks) {
        const double per_sm = (double)(pa.unit_blocks * LH) / p->n_sms;
        const double nt = (double)pa.unit_pairs / pa.unit_blocks, own = (double)own_tiles / pa.unit_blocks;
        whole = std::ceil(per_sm) * (nt + own + 1.7) <= per_sm * (1.15 * nt + 6.3) + 6.;
    }
    // Consecutive blocks of a CTA: one where the prefix is long, so that a unit's
    // blocks run side by side and read it once from DRAM (21 tiles: 925 us with runs
    // of 1, 936 of 4, 959 with one run; 47: 1,052, 1,080, 1,112); some 32 tiles'
    // worth where it is short and the next block's first loads count (4 tiles: 388
    // us with 1, 347 with 4, 338 with 8; 7: 846, 817, 804; 12: 268, 261, 262).
    pa.run = (int32_t)std::max<int64_t>(1, pa.unit_pairs > 0 ? 32 * pa.unit_blocks / pa.unit_pairs : 1);
    for (int g = 0; g < n_groups; ++g)
        for (int b = group_offsets[g]; b < group_offsets[g + 1]; ++b)
            pl.rq[b].group = place[g];
    pa.n_groups = n_groups;

    // slices whose partial results fit kMaxPartBytes
    int lh_slice = LH;
    if (pa.unit_blocks > 0 && !whole) {
        const int64_t fit = (kMaxPartBytes / kSharedPartBytes - p->n_sms) / pa.unit_blocks;
        const int64_t n = (LH + std::max<int64_t>(1, fit) - 1) / std::max<int64_t>(1, fit);
        lh_slice = (int)((LH + n - 1) / n);
    }
    kvr_status st;
    cudaError_t e;
    const int64_t q_rows = (int64_t)L * sa.total_q * Hq;
    if ((st = p->grow_query_scratch((size_t)q_rows * D * 2)) != KVR_OK ||
        (pa.unit_blocks > 0 && !whole &&
         (st = p->grow_part_scratch((size_t)(lh_slice * pa.unit_blocks + p->n_sms) * kSharedPartBytes)) != KVR_OK))
        return st;
    pa.part = static_cast<float *>(p->part);
    pa.q_rot = p->q_rot;
    // Own rows: each request's kernel by its own rows.  For those of long queries the row
    // groups of a (request, unit) that one CTA takes, as many as leave three CTAs per SM of
    // all the call's groups (63 single tokens and one query of 2,048, 8 units: 0.30 ms a
    // call, 7.1 where kernel and groups went by the longest query; 288 units: 10.6 and 17.0)
    auto own_groups = [&](const DevShared &r) -> int64_t {
        const int64_t rows = (int64_t)r.q_len * G;
        return rows > kOwnFewRows ? (rows + kOwnRowsMax - 1) / kOwnRowsMax : 0;
    };
    int64_t groups = 0, most = 1;
    int32_t few_rows = 0, max_own = 1;
    for (const DevShared &r : pl.rq) {
        const int64_t n = own_groups(r);
        groups += n;
        most = std::max(most, n);
        if (n > 0)
            max_own = std::max(max_own, r.own + r.q_len);
        else
            few_rows = std::max(few_rows, r.q_len * G);
    }
    const int64_t per_cta = std::min(most, std::max<int64_t>(1, groups * lh_slice / (3 * (int64_t)p->n_sms)));
    int64_t chunks = 0;
    for (DevShared &r : pl.rq) {
        r.chunk0 = (int32_t)chunks;   // (at most a chunk a query row: within 32 bits)
        chunks += (own_groups(r) + per_cta - 1) / per_cta;
    }
    CUtensorMap mq, mpk, mpv, mk, mv;
    if ((st = encode_rows_map(*p, p->q_rot, q_rows, 128, &mq)) != KVR_OK ||
        (any_prefix && ((st = encode_rows_map(*p, sa.prefix_k, pre_rows, 128, &mpk)) != KVR_OK ||
                        (st = encode_rows_map(*p, sa.prefix_v, pre_rows, 128, &mpv)) != KVR_OK)) ||
        (st = encode_rows_map(*p, sa.cache_k, own_rows, whole ? 128 : 32, &mk)) != KVR_OK ||
        (st = encode_rows_map(*p, sa.cache_v, own_rows, whole ? 128 : 32, &mv)) != KVR_OK)
        return st;
    // the previous call's attention must be done with the scratch
    if (p->q_rot_used && (e = cudaStreamWaitEvent(s, p->q_rot_done, 0)) != cudaSuccess)
        return cuda_fail(e, "query scratch ordering");
    Slot *slot = nullptr;
    if (sa.n_reqs <= kInlineEntries && n_groups <= kInlineEntries) {
        std::memcpy(pl.tab.reqs, pl.rq.data(), pl.rq.size() * sizeof(DevShared));
        std::memcpy(pl.gtab.groups, pl.gr.data(), pl.gr.size() * sizeof(DevGroup));
    } else {
        const size_t off = pl.rq.size() * sizeof(DevShared);
        std::vector<char> rows(off + pl.gr.size() * sizeof(DevGroup));
        std::memcpy(rows.data(), pl.rq.data(), off);
        std::memcpy(rows.data() + off, pl.gr.data(), pl.gr.size() * sizeof(DevGroup));
        if ((st = upload_table(p, rows.data(), rows.size(), s, &slot)) != KVR_OK)
            return st;
        sa.reqs = static_cast<const DevShared *>(slot->dev);
        pa.groups = reinterpret_cast<const DevGroup *>(static_cast<const char *>(slot->dev) + off);
    }
    SharedTcArgs t{&sa, &pl.tab, &pa, &pl.gtab, &mq, any_prefix ? &mpk : nullptr, any_prefix ? &mpv : nullptr,
                   &mk, &mv, p->n_sms, whole, few_rows, (int32_t)per_cta, (int32_t)chunks, max_own};
    p->shared_path = whole ? KVR_SHARED_WHOLE : KVR_SHARED_PARTS;
    p->mark(2, s);
    {
        NvtxRange r("kvr.k_shared_prologue");
        e = launch_shared_prologue(sa, pl.tab, p->q_rot, !p->timed, s);
    }
    p->mark(3, s);
    p->mark(4, s);
    for (int lh = 0; lh < LH && e == cudaSuccess; lh += lh_slice) {
        NvtxRange r("kvr.k_shared_prefix_own");
        pa.lh_base = lh;
        pa.lh_count = std::min(lh_slice, LH - lh);
        pa.total = pa.lh_count * (whole ? pa.unit_blocks : pa.unit_pairs);
        pa.n_ctas = (int32_t)std::min<int64_t>(p->n_sms, pa.total);
        pa.ratio = pa.total > 0 ? (float)((double)pa.n_ctas / (double)pa.total) : 0.f;
        e = launch_shared_tc(t, !p->timed, s);
    }
    p->mark(5, s);
    cudaEventRecord(p->q_rot_done, s);
    p->q_rot_used = true;
    if (slot)
        cudaEventRecord(slot->done, s);
    return e == cudaSuccess ? KVR_OK : cuda_fail(e, "shared-prefix attention launch");
}

}  // namespace

extern "C" kvr_status kvr_shared_query_attention(kvr_pool_t p, int32_t n_groups, const int32_t *group_offsets,
                                                 const int64_t *prefix_offsets, const int32_t *prefix_len,
                                                 const void *prefix_k, const void *prefix_v,
                                                 const int64_t *cache_offsets, const int32_t *own_len,
                                                 const int32_t *q_offsets, const void *q, const void *kq,
                                                 const void *vq, void *cache_k, void *cache_v, void *out,
                                                 float softmax_scale, void *stream)
{
    if (!p)
        return fail(KVR_ERR_INVALID_ARG, "pool is NULL");
    if (n_groups < 0)
        return fail(KVR_ERR_INVALID_ARG, "n_groups %d", n_groups);
    if (n_groups == 0)
        return KVR_OK;
    NvtxRange call("kvr_shared_query_attention");
    return guarded([&]() -> kvr_status {
        kvr_status st;
        if ((st = check_offsets32(group_offsets, n_groups, "group_offsets")) != KVR_OK)
            return st;
        const int32_t batch = group_offsets[n_groups];
        if (batch == 0)
            return KVR_OK;
        if ((st = check_cache_offsets(prefix_offsets, n_groups)) != KVR_OK ||
            (st = check_cache_offsets(cache_offsets, batch)) != KVR_OK ||
            (st = check_offsets32(q_offsets, batch, "q_offsets")) != KVR_OK)
            return st;
        if (!prefix_len || !own_len)
            return fail(KVR_ERR_INVALID_ARG, "prefix_len / own_len is NULL");
        if (!(softmax_scale >= 0.f) || !std::isfinite(softmax_scale))
            return fail(KVR_ERR_INVALID_ARG, "softmax_scale %g", (double)softmax_scale);
        bool any_prefix = false;
        for (int g = 0; g < n_groups; ++g) {
            if (prefix_len[g] < 0 || prefix_len[g] > prefix_offsets[g + 1] - prefix_offsets[g])
                return fail(KVR_ERR_OUT_OF_RANGE, "group %d: prefix %d rows outside its block of %lld", g, prefix_len[g],
                            (long long)(prefix_offsets[g + 1] - prefix_offsets[g]));
            any_prefix = any_prefix || prefix_len[g] > 0;
        }
        const int L = p->d.n_layers, H = p->d.n_kv_heads, Hq = p->d.n_q_heads, D = p->d.head_dim, LH = L * H;
        const int32_t T = q_offsets[batch];
        SharedPlan pl;
        pl.rq.reserve(batch);
        for (int g = 0; g < n_groups; ++g)
            for (int b = group_offsets[g]; b < group_offsets[g + 1]; ++b) {
                const int64_t cap = cache_offsets[b + 1] - cache_offsets[b];
                const int32_t lq = q_offsets[b + 1] - q_offsets[b];
                if (own_len[b] < 0 || (int64_t)own_len[b] + lq > cap)
                    return fail(KVR_ERR_OUT_OF_RANGE, "request %d: own rows %d + query %d > cache block %lld", b,
                                own_len[b], lq, (long long)cap);
                if ((int64_t)prefix_len[g] + own_len[b] + lq > kMaxPosition)
                    return fail(KVR_ERR_OUT_OF_RANGE, "request %d: positions beyond 2^24", b);
                DevShared r{};
                r.cache_row0 = cache_offsets[b] * LH;
                r.pre_row0 = prefix_offsets[g] * LH;
                r.cap = (int32_t)cap;
                r.own = own_len[b];
                r.pre_cap = (int32_t)(prefix_offsets[g + 1] - prefix_offsets[g]);
                r.pre_len = prefix_len[g];
                r.q_off = q_offsets[b];
                r.q_len = lq;
                pl.rq.push_back(r);
            }
        if (T == 0)
            return KVR_OK;
        const void *ptrs[] = {q, kq, vq, cache_k, cache_v, out};
        for (const void *x : ptrs)
            if (!x || !aligned16(x))
                return fail(KVR_ERR_INVALID_ARG, "q / kq / vq / cache / out NULL or not 16-byte aligned");
        if (any_prefix && (!prefix_k || !prefix_v || !aligned16(prefix_k) || !aligned16(prefix_v)))
            return fail(KVR_ERR_INVALID_ARG, "prefix_k / prefix_v NULL or not 16-byte aligned");
        const int64_t own_rows[2] = {cache_offsets[0] * LH, cache_offsets[batch] * LH};
        const int64_t pre_rows[2] = {prefix_offsets[0] * LH, prefix_offsets[n_groups] * LH};
        const int64_t row_bytes = (int64_t)D * p->elt();
        const Range dst[3] = {range_of(cache_k, own_rows[0], own_rows[1], row_bytes),
                              range_of(cache_v, own_rows[0], own_rows[1], row_bytes),
                              range_of(out, 0, (int64_t)L * T * Hq, row_bytes)};
        const Range src[2] = {range_of(prefix_k, pre_rows[0], pre_rows[1], row_bytes),
                              range_of(prefix_v, pre_rows[0], pre_rows[1], row_bytes)};
        for (const Range &d : dst)
            for (const Range &x : src)
                if (any_prefix && d.meets(x))
                    return fail(KVR_ERR_INVALID_ARG, "the cache or the output overlaps the shared prefix");
        for (int i = 0; i < 3; ++i)
            for (int j = 0; j < i; ++j)
                if (dst[i].meets(dst[j]))
                    return fail(KVR_ERR_INVALID_ARG, "the caches and the output overlap");
        // the queries' keys and values are appended, and rows of the output written, while
        // other rows of the inputs are still read (each row of q only before its own output)
        const Range in[3] = {range_of(q, 0, (int64_t)L * T * Hq, row_bytes), range_of(kq, 0, (int64_t)L * T * H, row_bytes),
                             range_of(vq, 0, (int64_t)L * T * H, row_bytes)};
        for (const Range &x : in)
            if (x.meets(dst[0]) || x.meets(dst[1]))
                return fail(KVR_ERR_INVALID_ARG, "the caches overlap the query inputs");
        if (in[0].meets(dst[2]) && in[0].lo != dst[2].lo)
            return fail(KVR_ERR_INVALID_ARG, "the output overlaps the queries (it may only be the same buffer)");
        cudaStream_t s = static_cast<cudaStream_t>(stream);
        const bool may_tc = attention_tc_supported(p->d.dtype, D);
        if ((st = check_capture(*p, s, !may_tc && batch <= kInlineEntries,
                                "the call uses library scratch, or uploads the tables of more than 64 requests")) != KVR_OK ||
            (st = ensure_device(p)) != KVR_OK)
            return st;
        DeviceGuard g(p->device);
        const bool tc = use_tensor_cores(*p);
        if (tc && std::max({own_rows[1], pre_rows[1], (int64_t)L * T * Hq}) > (int64_t)INT32_MAX - 256)
            return fail(KVR_ERR_UNSUPPORTED, "cache, prefix or query rows exceed the int32 TMA coordinate range");
        SharedArgs sa{};
        sa.rope = p->rope;
        sa.q = q;
        sa.kq = kq;
        sa.vq = vq;
        sa.prefix_k = prefix_k;
        sa.prefix_v = prefix_v;
        sa.cache_k = cache_k;
        sa.cache_v = cache_v;
        sa.out = out;
        sa.n_reqs = batch;
        sa.n_layers = L;
        sa.n_q_heads = Hq;
        sa.n_kv_heads = H;
        sa.total_q = T;
        sa.scale_log2 = (softmax_scale > 0.f ? softmax_scale : 1.f / std::sqrt((float)D)) * 1.4426950408889634f;
        sa.interleaved = (p->d.flags & KVR_POOL_ROPE_INTERLEAVED) ? 1 : 0;
        sa.err = p->err;
        if (tc)
            return shared_tc(p, pl, sa, n_groups, group_offsets, prefix_offsets, prefix_len, any_prefix, q_offsets,
                             own_rows[1], pre_rows[1], s);
        return shared_simt(p, pl, sa, s);
    });
}

extern "C" kvr_status kvr_key_weights(kvr_pool_t p, int32_t batch, const int64_t *cache_offsets,
                                      const int32_t *prefix_len, const int32_t *q_offsets, const void *q,
                                      const void *cache_k, float *weights, float softmax_scale, uint32_t flags,
                                      void *stream)
{
    if (!p)
        return fail(KVR_ERR_INVALID_ARG, "pool is NULL");
    if (batch < 0)
        return fail(KVR_ERR_INVALID_ARG, "batch %d", batch);
    if (flags & ~(uint32_t)KVR_WEIGHTS_ACCUMULATE)
        return fail(KVR_ERR_INVALID_ARG, "unknown flags 0x%x", flags);
    if (batch == 0)
        return KVR_OK;
    NvtxRange call("kvr_key_weights");
    return guarded([&]() -> kvr_status {
        kvr_status st;
        if ((st = check_cache_offsets(cache_offsets, batch)) != KVR_OK ||
            (st = check_offsets32(q_offsets, batch, "q_offsets")) != KVR_OK)
            return st;
        if (!prefix_len)
            return fail(KVR_ERR_INVALID_ARG, "prefix_len is NULL");
        if (!(softmax_scale >= 0.f) || !std::isfinite(softmax_scale))
            return fail(KVR_ERR_INVALID_ARG, "softmax_scale %g", (double)softmax_scale);
        const int L = p->d.n_layers, H = p->d.n_kv_heads, Hq = p->d.n_q_heads, D = p->d.head_dim, LH = L * H;
        const int32_t T = q_offsets[batch];
        const bool accumulate = flags & KVR_WEIGHTS_ACCUMULATE;
        std::vector<DevReq> rq(batch);
        WeightsArgs a{};
        for (int b = 0; b < batch; ++b) {
            const int64_t cap = cache_offsets[b + 1] - cache_offsets[b];
            const int32_t lq = q_offsets[b + 1] - q_offsets[b];
            if (prefix_len[b] < 0 || (int64_t)prefix_len[b] + lq > cap)
                return fail(KVR_ERR_OUT_OF_RANGE, "request %d: prefix %d + query %d > cache block %lld", b, prefix_len[b],
                            lq, (long long)cap);
            rq[b] = DevReq{};
            rq[b].cache_row0 = cache_offsets[b] * LH;
            rq[b].cap = (int32_t)cap;
            rq[b].prefix = prefix_len[b];
            rq[b].q_off = q_offsets[b];
            rq[b].q_len = lq;
            a.max_rows = std::max(a.max_rows, prefix_len[b] + lq);
            a.max_q_len = std::max(a.max_q_len, lq);
        }
        if (a.max_rows == 0 || (T == 0 && accumulate))
            return KVR_OK;
        if (!cache_k || !aligned16(cache_k) || (T > 0 && (!q || !aligned16(q))))
            return fail(KVR_ERR_INVALID_ARG, "q / cache_k NULL or not 16-byte aligned");
        if (!weights || (reinterpret_cast<uintptr_t>(weights) & 3))
            return fail(KVR_ERR_INVALID_ARG, "weights NULL or not 4-byte aligned");
        const int64_t r0 = cache_offsets[0] * LH, r1 = cache_offsets[batch] * LH, row_bytes = (int64_t)D * p->elt();
        const Range wr = range_of(weights, r0, r1, 4);
        if (wr.meets(range_of(cache_k, r0, r1, row_bytes)) ||
            (T > 0 && wr.meets(range_of(q, 0, (int64_t)L * T * Hq, row_bytes))))
            return fail(KVR_ERR_INVALID_ARG, "weights overlap the cache or the queries");
        cudaStream_t s = static_cast<cudaStream_t>(stream);
        const bool inl = batch <= kInlineEntries;
        if ((st = check_capture(*p, s, inl, "a call of more than 64 requests uploads its tables")) != KVR_OK ||
            (st = ensure_device(p)) != KVR_OK)
            return st;
        DeviceGuard g(p->device);
        a.rope = p->rope;
        a.q = q;
        a.cache_k = cache_k;
        a.weights = weights;
        a.n_reqs = batch;
        a.n_layers = L;
        a.n_q_heads = Hq;
        a.n_kv_heads = H;
        a.total_q = T;
        a.scale_log2 = (softmax_scale > 0.f ? softmax_scale : 1.f / std::sqrt((float)D)) * 1.4426950408889634f;
        a.interleaved = (p->d.flags & KVR_POOL_ROPE_INTERLEAVED) ? 1 : 0;
        a.accumulate = accumulate ? 1 : 0;
        a.err = p->err;
        // the tensor cores' TMA coordinates are 32-bit rows
        const bool tc = use_tensor_cores(*p) && r1 <= (int64_t)INT32_MAX - 256;
        CUtensorMap mk;
        if (tc && (st = encode_cache_map(*p, const_cast<void *>(cache_k), r1, &mk)) != KVR_OK)
            return st;
        // On the tensor cores each request goes to the kernel for its own query rows, a
        // launch for those of either (63 single tokens and a window of 64 on 1,200 keys, 288
        // units: 1.00 ms, 1.48 with all in the window's kernel, which reads K twice; 15 and
        // one on 16,000, 64 units: 0.89 and 1.65; 16 requests of 7 to 84 rows: 192 us, 187)
        int32_t few = batch;
        if (tc)
            few = (int32_t)(std::stable_partition(rq.begin(), rq.end(),
                                                  [&](const DevReq &r) { return (int64_t)r.q_len * (Hq / H) <= kWeightsFewRows; }) -
                            rq.begin());
        ReqTable tab;
        Slot *slot = nullptr;
        if (inl) {
            std::memcpy(tab.reqs, rq.data(), rq.size() * sizeof(DevReq));
        } else {
            if ((st = upload_table(p, rq.data(), rq.size() * sizeof(DevReq), s, &slot)) != KVR_OK)
                return st;
            a.reqs = static_cast<const DevReq *>(slot->dev);
        }
        cudaError_t e = cudaSuccess;
        NvtxRange r("kvr.k_key_weights");
        if (!tc)
            e = launch_weights_simt(a, tab, p->d.dtype, D, p->n_sms, s);
        for (int part = 0; tc && part < 2 && e == cudaSuccess; ++part) {
            a.req0 = part ? few : 0;
            a.n_reqs = part ? batch - few : few;
            a.max_rows = a.max_q_len = 0;
            for (int i = a.req0; i < a.req0 + a.n_reqs; ++i) {
                a.max_rows = std::max(a.max_rows, rq[i].prefix + rq[i].q_len);
                a.max_q_len = std::max(a.max_q_len, rq[i].q_len);
            }
            if (a.max_rows > 0)
                e = launch_weights_tc(a, tab, &mk, p->n_sms, s);
        }
        if (slot)
            cudaEventRecord(slot->done, s);
        return e == cudaSuccess ? KVR_OK : cuda_fail(e, "key weights launch");
    });
}

extern "C" kvr_status kvr_evict(kvr_pool_t p, int32_t batch, const int64_t *cache_offsets, const int32_t *kv_len,
                                const int32_t *keep, int32_t n_first, int32_t n_recent, const float *weights,
                                const void *cache_k, const void *cache_v, const int64_t *dst_offsets, void *dst_k,
                                void *dst_v, float *dst_weights, int32_t *kept, uint32_t flags, void *stream)
{
    if (!p)
        return fail(KVR_ERR_INVALID_ARG, "pool is NULL");
    if (batch < 0)
        return fail(KVR_ERR_INVALID_ARG, "batch %d", batch);
    if (flags & ~(uint32_t)KVR_EVICT_KEEP_ROTATION)
        return fail(KVR_ERR_INVALID_ARG, "unknown flags 0x%x", flags);
    if (n_first < 0 || n_recent < 0)
        return fail(KVR_ERR_INVALID_ARG, "n_first %d, n_recent %d", n_first, n_recent);
    if (batch == 0)
        return KVR_OK;
    NvtxRange call("kvr_evict");
    return guarded([&]() -> kvr_status {
        kvr_status st;
        if ((st = check_cache_offsets(cache_offsets, batch)) != KVR_OK ||
            (st = check_cache_offsets(dst_offsets, batch)) != KVR_OK)
            return st;
        if (!kv_len || !keep)
            return fail(KVR_ERR_INVALID_ARG, "kv_len / keep is NULL");
        const int LH = p->d.n_layers * p->d.n_kv_heads, D = p->d.head_dim;
        std::vector<DevEvict> rq(batch);
        EvictArgs a{};
        int64_t kept0 = 0, chunks = 0;
        for (int b = 0; b < batch; ++b) {
            const int64_t cap = cache_offsets[b + 1] - cache_offsets[b], dcap = dst_offsets[b + 1] - dst_offsets[b];
            if (kv_len[b] < 0 || kv_len[b] > cap)
                return fail(KVR_ERR_OUT_OF_RANGE, "request %d: %d rows outside its block of %lld", b, kv_len[b],
                            (long long)cap);
            if (keep[b] < 0 || (int64_t)n_first + n_recent > keep[b])
                return fail(KVR_ERR_INVALID_ARG, "request %d: keep %d < n_first %d + n_recent %d", b, keep[b], n_first,
                            n_recent);
            const int32_t k = std::min(keep[b], kv_len[b]);
            if (k > dcap)
                return fail(KVR_ERR_OUT_OF_RANGE, "request %d: %d kept rows > destination block %lld", b, k,
                            (long long)dcap);
            DevEvict r{};
            r.src_row0 = cache_offsets[b] * LH;
            r.dst_row0 = dst_offsets[b] * LH;
            r.kept0 = kept0;
            r.src_cap = (int32_t)cap;
            r.dst_cap = (int32_t)dcap;
            r.n = kv_len[b];
            r.keep = k;
            r.chunk0 = (int32_t)std::min<int64_t>(chunks, INT32_MAX);
            rq[b] = r;
            kept0 += (int64_t)k * LH;
            chunks += (int64_t)LH * std::max(1, (k + kEvictChunk - 1) / kEvictChunk);
            a.max_n = std::max(a.max_n, kv_len[b]);
            a.max_keep = std::max(a.max_keep, k);
        }
        if (chunks > INT32_MAX)
            return fail(KVR_ERR_UNSUPPORTED, "too many rows to move in one call");
        const int64_t s0 = cache_offsets[0] * LH, s1 = cache_offsets[batch] * LH;
        const int64_t d0 = dst_offsets[0] * LH, d1 = dst_offsets[batch] * LH, row_bytes = (int64_t)D * p->elt();
        if (s0 == s1 && d0 == d1)
            return KVR_OK;
        if (s0 < s1 && (!cache_k || !cache_v || !weights || !aligned16(cache_k) || !aligned16(cache_v)))
            return fail(KVR_ERR_INVALID_ARG, "cache_k / cache_v NULL or not 16-byte aligned, or weights NULL");
        if (kept0 > 0 && (!dst_k || !dst_v || !kept || !aligned16(dst_k) || !aligned16(dst_v)))
            return fail(KVR_ERR_INVALID_ARG, "dst_k / dst_v NULL or not 16-byte aligned, or kept NULL");
        if ((reinterpret_cast<uintptr_t>(weights) & 3) || (reinterpret_cast<uintptr_t>(dst_weights) & 3) ||
            (reinterpret_cast<uintptr_t>(kept) & 3))
            return fail(KVR_ERR_INVALID_ARG, "weights / dst_weights / kept not 4-byte aligned");
        // each destination is apart from everything else, or is its own source, block for block
        const bool same = std::equal(cache_offsets, cache_offsets + batch + 1, dst_offsets);
        const Range src[3] = {range_of(cache_k, s0, s1, row_bytes), range_of(cache_v, s0, s1, row_bytes),
                              range_of(weights, s0, s1, 4)};
        const Range dst[4] = {range_of(dst_k, d0, d1, row_bytes), range_of(dst_v, d0, d1, row_bytes),
                              range_of(dst_weights, d0, d1, 4), range_of(kept, 0, kept0, 4)};
        for (int i = 0; i < 4; ++i) {
            for (int j = 0; j < 3; ++j) {
                if (i == j && same && dst[i].lo == src[j].lo) {
                    if (dst[i].meets(src[j]))
                        a.in_place = 1;
                } else if (dst[i].meets(src[j])) {
                    return fail(KVR_ERR_INVALID_ARG, "a destination overlaps a source (only the same block is evicted in place)");
                }
            }
            for (int j = 0; j < i; ++j)
                if (dst[i].meets(dst[j]))
                    return fail(KVR_ERR_INVALID_ARG, "destinations overlap");
        }
        cudaStream_t s = static_cast<cudaStream_t>(stream);
        const bool inl = batch <= kInlineEntries;
        if ((st = check_capture(*p, s, inl, "a call of more than 64 requests uploads its tables")) != KVR_OK ||
            (st = ensure_device(p)) != KVR_OK)
            return st;
        DeviceGuard g(p->device);
        a.rope = p->rope;
        a.rope_turns = p->rope_turns;
        a.weights = weights;
        a.cache_k = cache_k;
        a.cache_v = cache_v;
        a.dst_k = dst_k;
        a.dst_v = dst_v;
        a.dst_weights = dst_weights;
        a.kept = kept;
        a.n_reqs = batch;
        a.units = LH;
        a.n_first = n_first;
        a.n_recent = n_recent;
        a.n_chunks = (int32_t)chunks;
        a.interleaved = (p->d.flags & KVR_POOL_ROPE_INTERLEAVED) ? 1 : 0;
        a.keep_rotation = (flags & KVR_EVICT_KEEP_ROTATION) ? 1 : 0;
        EvictTable tab;
        Slot *slot = nullptr;
        if (inl) {
            std::memcpy(tab.reqs, rq.data(), rq.size() * sizeof(DevEvict));
        } else {
            if ((st = upload_table(p, rq.data(), rq.size() * sizeof(DevEvict), s, &slot)) != KVR_OK)
                return st;
            a.reqs = static_cast<const DevEvict *>(slot->dev);
        }
        cudaError_t e;
        {
            NvtxRange r("kvr.k_evict");
            e = launch_evict(a, tab, p->d.dtype, D, p->n_sms, s);
        }
        if (slot)
            cudaEventRecord(slot->done, s);
        return e == cudaSuccess ? KVR_OK : cuda_fail(e, "eviction launch");
    });
}

// ---------------------------------------------------------------------------
// paged cache
// ---------------------------------------------------------------------------
namespace {

// One call: its requests and the page numbers that its kernels read.
struct PagePlan {
    std::vector<DevPageReq> rq;
    std::vector<int32_t> ids;
    PageTable tab;
    PageArgs a{};
    Slot *slot = nullptr;
    bool inl() const { return rq.size() <= (size_t)kInlineEntries && ids.size() <= (size_t)kInlinePages; }
};

// Elements from a page pool's first element to behind its last row.
int64_t page_extent(const kvr_pool &p, const kvr_pages &g)
{
    return (g.n_pages - 1) * g.stride[0] + (p.d.n_layers - 1) * g.stride[1] + (p.d.n_kv_heads - 1) * g.stride[2] +
           (int64_t)g.page_rows * p.d.head_dim;
}

// Whether runs of `run` bytes at the sums of `n` strides (ascending, each at least what the ones before
// it span) meet the same ones `d` bytes further on.  Within its stride's multiples an outer distance is
// made good by the nearest two: what the inner ones span is at most one stride.
bool runs_meet(int64_t d, const int64_t *stride, const int64_t *count, int n, int64_t run)
{
    if (n == 0)
        return -run < d && d < run;
    const int64_t s = stride[n - 1], j0 = d / s;
    for (int64_t j = j0 - 1; j <= j0 + 1; ++j)
        if (-count[n - 1] < j && j < count[n - 1] && runs_meet(d - j * s, stride, count, n - 1, run))
            return true;
    return false;
}

// `written`: the call writes rows, which must then not lie upon each other.
kvr_status check_pages(const kvr_pool &p, const kvr_pages *pages, bool written)
{
    if (!pages)
        return fail(KVR_ERR_INVALID_ARG, "pages is NULL");
    const kvr_pages &g = *pages;
    if (g.n_pages < 1 || g.n_pages > INT32_MAX || g.page_rows < 1 || g.page_rows > kMaxPosition)
        return fail(KVR_ERR_INVALID_ARG, "n_pages %lld, page_rows %d", (long long)g.n_pages, g.page_rows);
    if (!g.k || !g.v || !aligned16(g.k) || !aligned16(g.v))
        return fail(KVR_ERR_INVALID_ARG, "pages: k / v NULL or not 16-byte aligned");
    const int64_t count[3] = {g.n_pages, p.d.n_layers, p.d.n_kv_heads};
    for (int i = 0; i < 3; ++i)
        if (g.stride[i] < 0 || g.stride[i] % p.vec_elems() || g.stride[i] > (int64_t(1) << 58) / count[i])
            return fail(KVR_ERR_INVALID_ARG, "pages: stride[%d] = %lld must be >= 0, a multiple of %d and within 2^58 elements", i,
                        (long long)g.stride[i], p.vec_elems());
    if (written) {
        if (g.k == g.v)
            return fail(KVR_ERR_INVALID_ARG, "pages: k and v are the same rows, of which the call writes both");
        int o[3] = {0, 1, 2};
        std::sort(o, o + 3, [&](int x, int y) { return g.stride[x] < g.stride[y]; });
        int64_t need = (int64_t)g.page_rows * p.d.head_dim;
        for (int i : o) {
            if (count[i] > 1 && g.stride[i] < need)
                return fail(KVR_ERR_INVALID_ARG, "pages: stride[%d] = %lld lays rows upon each other", i, (long long)g.stride[i]);
            if (count[i] > 1)
                need = (count[i] - 1) * g.stride[i] + need;
        }
        int64_t stride[3], number[3];
        int n = 0;
        for (int i : o)
            if (count[i] > 1) {
                stride[n] = g.stride[i] * p.elt();
                number[n++] = count[i];
            }
        // (apart as a whole, as in most caches: their distance may be beyond 2^63)
        if (range_of(g.k, 0, need, p.elt()).meets(range_of(g.v, 0, need, p.elt())) &&
            runs_meet((int64_t)(reinterpret_cast<uintptr_t>(g.v) - reinterpret_cast<uintptr_t>(g.k)), stride, number, n,
                      (int64_t)g.page_rows * p.d.head_dim * p.elt()))
            return fail(KVR_ERR_INVALID_ARG, "pages: rows of v lie upon rows of k, and the call writes both");
    }
    return KVR_OK;
}

kvr_status check_packed(const kvr_pool &p, const kvr_packed_pages *packed, int32_t page_rows)
{
    if (!packed)
        return fail(KVR_ERR_INVALID_ARG, "packed is NULL");
    if (p.d.dtype != KVR_DTYPE_BF16 || p.d.head_dim != 128)
        return fail(KVR_ERR_UNSUPPORTED, "packed pages need a bf16 pool with head_dim 128");
    if (!packed->data || !aligned16(packed->data))
        return fail(KVR_ERR_INVALID_ARG, "packed: data NULL or not 16-byte aligned");
    if (packed->n_pages < 1 || packed->n_pages > INT32_MAX)
        return fail(KVR_ERR_INVALID_ARG, "packed: n_pages %lld", (long long)packed->n_pages);
    if (page_rows % kPackRows)
        return fail(KVR_ERR_INVALID_ARG, "packed pages: page_rows %d must be a multiple of %d", page_rows, kPackRows);
    if ((double)packed->n_pages * p.d.n_layers * p.d.n_kv_heads * (page_rows / kPackRows) * kPackBytes > 1e18)
        return fail(KVR_ERR_INVALID_ARG, "packed: %lld pages of %d rows", (long long)packed->n_pages, page_rows);
    return KVR_OK;
}

int64_t packed_page_bytes(const kvr_pool &p, int32_t page_rows)
{
    return (int64_t)p.d.n_layers * p.d.n_kv_heads * (page_rows / kPackRows) * kPackBytes;
}

Range pages_range(const kvr_pool &p, const kvr_pages &g, bool values)
{
    return range_of(values ? g.v : g.k, 0, page_extent(p, g), p.elt());
}
Range packed_range(const kvr_pool &p, const kvr_packed_pages &k, int32_t page_rows)
{
    return range_of(k.data, 0, k.n_pages, packed_page_bytes(p, page_rows));
}

// Appends pages [g0, g1) of request b to the list.
kvr_status take_pages(std::vector<int32_t> &ids, const int32_t *table, int64_t width, int b, int64_t g0, int64_t g1, int64_t n_pages,
                      const char *what)
{
    if (g0 >= g1)
        return KVR_OK;
    if (!table)
        return fail(KVR_ERR_INVALID_ARG, "%s table is NULL", what);
    if (g1 > width)
        return fail(KVR_ERR_OUT_OF_RANGE, "request %d: page %lld outside its %s table of %lld", b, (long long)(g1 - 1), what,
                    (long long)width);
    const int32_t *row = table + (int64_t)b * width;
    for (int64_t g = g0; g < g1; ++g)
        if (row[g] < 0 || row[g] >= n_pages)
            return fail(KVR_ERR_OUT_OF_RANGE, "request %d: page %lld is %d, of %lld %s pages", b, (long long)g, row[g],
                        (long long)n_pages, what);
    ids.insert(ids.end(), row + g0, row + g1);
    return KVR_OK;
}

// A page that a call writes must be in its list once.
kvr_status check_distinct(const std::vector<int32_t> &ids, size_t from)
{
    std::vector<int32_t> x(ids.begin() + from, ids.end());
    std::sort(x.begin(), x.end());
    const auto d = std::adjacent_find(x.begin(), x.end());
    if (d != x.end())
        return fail(KVR_ERR_INVALID_ARG, "page %d is written for two requests, or twice for one", *d);
    return KVR_OK;
}

void page_base(const kvr_pool &p, const kvr_pages &g, PagePlan &pl)
{
    PageArgs &a = pl.a;
    a.n_reqs = (int32_t)pl.rq.size();
    a.n_layers = p.d.n_layers;
    a.n_q_heads = p.d.n_q_heads;
    a.n_kv_heads = p.d.n_kv_heads;
    a.interleaved = (p.d.flags & KVR_POOL_ROPE_INTERLEAVED) ? 1 : 0;
    a.rope = p.rope;
    a.err = p.err;
    a.g.k = g.k;
    a.g.v = g.v;
    a.g.s_page = g.stride[0];
    a.g.s_layer = g.stride[1];
    a.g.s_head = g.stride[2];
    a.g.rows = g.page_rows;
    a.g.shift = (g.page_rows & (g.page_rows - 1)) == 0 ? __builtin_ctz((unsigned)g.page_rows) : -1;
}

// The plan's tables into its kernels' parameters, or uploaded.
kvr_status page_stage(kvr_pool *p, PagePlan &pl, cudaStream_t s)
{
    if (pl.inl()) {
        std::memcpy(pl.tab.reqs, pl.rq.data(), pl.rq.size() * sizeof(DevPageReq));
        if (!pl.ids.empty())
            std::memcpy(pl.tab.ids, pl.ids.data(), pl.ids.size() * sizeof(int32_t));
        return KVR_OK;
    }
    const size_t off = pl.rq.size() * sizeof(DevPageReq), bytes = off + pl.ids.size() * sizeof(int32_t);
    kvr_status st;
    if ((st = p->acquire(bytes, bytes, &pl.slot)) != KVR_OK)
        return st;
    char *h = static_cast<char *>(pl.slot->host);
    std::memcpy(h, pl.rq.data(), off);
    std::memcpy(h + off, pl.ids.data(), bytes - off);
    const cudaError_t e = cudaMemcpyAsync(pl.slot->dev, h, bytes, cudaMemcpyHostToDevice, s);
    cudaEventRecord(pl.slot->done, s);
    pl.slot->used = true;
    if (e != cudaSuccess)
        return cuda_fail(e, "table upload");
    pl.a.reqs = static_cast<const DevPageReq *>(pl.slot->dev);
    pl.a.ids = reinterpret_cast<const int32_t *>(static_cast<const char *>(pl.slot->dev) + off);
    return KVR_OK;
}

kvr_status page_ready(kvr_pool *p, const PagePlan &pl, cudaStream_t s)
{
    kvr_status st;
    if ((st = check_capture(*p, s, pl.inl(), "the call uploads the tables of more than 64 requests or 1,024 pages")) != KVR_OK ||
        (st = ensure_device(p)) != KVR_OK)
        return st;
    return KVR_OK;
}

// The tensor-core kernel's items: 256-row blocks of the requests of more than
// kPageFewRows query rows, each in `splits` stretches of its key tiles; and the slices
// of the units whose restored rows fit kMaxPartBytes.
kvr_status page_tc_plan(const kvr_pool *p, PagePlan &pl, const kvr_pages &g, int32_t window, int32_t n_first, PageTcArgs &tc, int &lh_slice)
{
    const int D = p->d.head_dim, G = p->d.n_q_heads / p->d.n_kv_heads, LH = p->d.n_layers * p->d.n_kv_heads;
    // boxes of the largest power of two of rows that no page boundary cuts; with a window at most 64, as
    // the first rows and the window's are rounded out to boxes (pages of 256 rows, 4,096-token prompt, 64
    // units: window 1,024 with 64 first rows 506 us, 550 with boxes of 128; with none 519 and 512; window
    // 200 with 4 first rows 326 and 382.  Boxes of 32 take the first to 529)
    tc.box = window > 0 ? 64 : 128;
    while (g.page_rows % tc.box)
        tc.box /= 2;
    if (tc.box < 16 || g.stride[0] % D || g.stride[1] % D || g.stride[2] % D || page_extent(*p, g) / D > (int64_t)INT32_MAX - 256)
        tc.box = 0;
    int64_t blocks = 0, tiles = 0, rest = 0;
    tc.one_tile = 1;
    for (DevPageReq &r : pl.rq) {
        r.tile0 = (int32_t)rest;
        if (r.q_len * (int64_t)G <= kPageFewRows)
            continue;
        if (r.q_len * (int64_t)G > INT32_MAX - 256)
            return fail(KVR_ERR_UNSUPPORTED, "too many query rows");
        const int64_t n = (r.q_len * (int64_t)G + 255) / 256;
        tc.one_tile = tc.one_tile && r.q_len * (int64_t)G <= 128;
        const int32_t hi = std::min<int32_t>(r.kv_len, r.pos0 + r.q_len);
        const int32_t lo = std::min(hi, window > 0 ? std::max(0, r.pos0 - window + 1) : 0);
        const int64_t seen = window > 0 ? std::min<int64_t>(hi, (int64_t)window + n_first + 256 / G) : hi;
        blocks += n;
        tiles += n * ((seen + 127) / 128);
        const page::RestTiles t = page::rest_tiles(hi, lo, std::min(n_first, lo), r.packed_len);
        if (r.packed_len > 0)
            rest += t.first + std::max(0, t.end - t.win);
        if (rest > (INT32_MAX - 256) / 128)
            return fail(KVR_ERR_UNSUPPORTED, "too many packed rows for queries of more than 16 rows");
    }
    tc.unit_tiles = (int32_t)rest;
    lh_slice = LH;
    if (rest > 0) {
        const int64_t fit = std::max<int64_t>(1, kMaxPartBytes / (rest * kPageTileBytes * 2)), n = (LH + fit - 1) / fit;
        lh_slice = (int)((LH + n - 1) / n);
    }
    // The time of a slice in units of a key tile (1.45 us): rounds of items, each its tiles
    // and 3 more, and for partial results 4 more and their traffic (266 KB an item).
    const double nt = (double)tiles / (double)std::max<int64_t>(1, blocks);
    double best = 1e30;
    for (int sp = 1; sp <= 32 && (sp == 1 || nt / sp >= 4.); ++sp) {
        const double items = (double)(blocks * lh_slice) * sp;
        const double t = std::ceil(items / p->n_sms) * (nt / sp + 3.) + (sp > 1 ? 4. + items * 266e3 / 6e6 / 1.45 : 0.);
        if (t < 0.97 * best) {
            best = t;
            tc.splits = sp;
        }
    }
    if (blocks * tc.splits > INT32_MAX)
        return fail(KVR_ERR_UNSUPPORTED, "too many query rows");
    int32_t item = 0;
    for (DevPageReq &r : pl.rq) {
        r.item0 = item;
        if (r.q_len * (int64_t)G > kPageFewRows)
            item += (int32_t)((r.q_len * (int64_t)G + 255) / 256) * tc.splits;
    }
    tc.unit_items = item;
    return KVR_OK;
}

// kvr_page_pack and kvr_page_unpack.
kvr_status page_pack(kvr_pool_t p, const kvr_pages *pages, const int32_t *table, const kvr_packed_pages *packed,
                     const int32_t *packed_table, int32_t batch, int32_t width, int32_t packed_width, const int32_t *begin,
                     const int32_t *end, bool unpack, void *stream)
{
    if (!p)
        return fail(KVR_ERR_INVALID_ARG, "pool is NULL");
    if (batch < 0 || width < 0 || packed_width < 0)
        return fail(KVR_ERR_INVALID_ARG, "batch %d, widths %d, %d", batch, width, packed_width);
    NvtxRange call(unpack ? "kvr_page_unpack" : "kvr_page_pack");
    return guarded([&]() -> kvr_status {
        kvr_status st;
        if ((st = check_pages(*p, pages, unpack)) != KVR_OK || (st = check_packed(*p, packed, pages->page_rows)) != KVR_OK)
            return st;
        if (batch > 0 && (!begin || !end))
            return fail(KVR_ERR_INVALID_ARG, "begin / end is NULL");
        const int32_t R = pages->page_rows;
        PagePlan pl;
        pl.rq.reserve(batch);
        int64_t blocks = 0;
        for (int b = 0; b < batch; ++b) {
            if (begin[b] < 0 || end[b] < begin[b] || end[b] > kMaxPosition || begin[b] % kPackRows || end[b] % kPackRows)
                return fail(KVR_ERR_INVALID_ARG, "request %d: rows %d to %d are not whole blocks of %d", b, begin[b], end[b], kPackRows);
            DevPageReq r{};
            r.pos0 = begin[b];
            r.q_off = (int32_t)blocks;
            r.q_len = (end[b] - begin[b]) / kPackRows;
            blocks += r.q_len;
            if (blocks > INT32_MAX)
                return fail(KVR_ERR_OUT_OF_RANGE, "more than 2^31 blocks");
            r.few = r.pfew = INT32_MAX;
            pl.rq.push_back(r);
        }
        for (int which = 0; which < 2; ++which) {   // the pages, then the packed ones
            const size_t from = pl.ids.size();
            for (int b = 0; b < batch; ++b) {
                const int64_t g0 = begin[b] / R, g1 = begin[b] < end[b] ? (end[b] + R - 1) / R : g0;
                (which ? pl.rq[b].poff : pl.rq[b].off)[0] = (int32_t)((int64_t)pl.ids.size() - g0);
                if ((st = which ? take_pages(pl.ids, packed_table, packed_width, b, g0, g1, packed->n_pages, "packed")
                                : take_pages(pl.ids, table, width, b, g0, g1, pages->n_pages, "page")) != KVR_OK)
                    return st;
            }
            if (which == (unpack ? 0 : 1) && (st = check_distinct(pl.ids, from)) != KVR_OK)
                return st;
        }
        if (pl.ids.size() > INT32_MAX)
            return fail(KVR_ERR_OUT_OF_RANGE, "too many pages");
        const Range pr = packed_range(*p, *packed, R);
        if (pr.meets(pages_range(*p, *pages, false)) || pr.meets(pages_range(*p, *pages, true)))
            return fail(KVR_ERR_INVALID_ARG, "the packed pages overlap the pages");
        if (blocks == 0)
            return KVR_OK;
        cudaStream_t s = static_cast<cudaStream_t>(stream);
        if ((st = page_ready(p, pl, s)) != KVR_OK)
            return st;
        DeviceGuard g(p->device);
        page_base(*p, *pages, pl);
        pl.a.g.packed = static_cast<uint8_t *>(packed->data);
        pl.a.g.packed_page = packed_page_bytes(*p, R);
        if ((st = page_stage(p, pl, s)) != KVR_OK)
            return st;
        NvtxRange r("kvr.k_page_pack");
        const cudaError_t e = launch_page_pack(pl.a, pl.tab, blocks, unpack, s);
        if (pl.slot)
            cudaEventRecord(pl.slot->done, s);
        return e == cudaSuccess ? KVR_OK : cuda_fail(e, unpack ? "unpack launch" : "pack launch");
    });
}

}  // namespace

extern "C" int64_t kvr_packed_page_bytes(kvr_pool_t p, int32_t page_rows)
{
    return p && p->d.dtype == KVR_DTYPE_BF16 && p->d.head_dim == 128 && page_rows > 0 && page_rows <= kMaxPosition &&
                   page_rows % kPackRows == 0
               ? packed_page_bytes(*p, page_rows)
               : 0;
}

extern "C" kvr_status kvr_page_append(kvr_pool_t p, const kvr_pages *pages, int32_t batch, const int32_t *table, int32_t width,
                                      const int32_t *start, const int32_t *q_offsets, const void *k, const void *v,
                                      const int64_t *stride, uint32_t flags, void *stream)
{
    if (!p)
        return fail(KVR_ERR_INVALID_ARG, "pool is NULL");
    if (batch < 0 || width < 0)
        return fail(KVR_ERR_INVALID_ARG, "batch %d, width %d", batch, width);
    if (flags & ~KVR_APPEND_TURNED)
        return fail(KVR_ERR_INVALID_ARG, "unknown flags 0x%x", flags);
    NvtxRange call("kvr_page_append");
    return guarded([&]() -> kvr_status {
        kvr_status st;
        if ((st = check_pages(*p, pages, true)) != KVR_OK || (st = check_offsets32(q_offsets, batch, "q_offsets")) != KVR_OK)
            return st;
        if (batch > 0 && !start)
            return fail(KVR_ERR_INVALID_ARG, "start is NULL");
        const int L = p->d.n_layers, H = p->d.n_kv_heads, D = p->d.head_dim;
        const int32_t T = q_offsets[batch], R = pages->page_rows;
        PagePlan pl;
        pl.rq.reserve(batch);
        for (int b = 0; b < batch; ++b) {
            DevPageReq r{};
            r.q_off = q_offsets[b];
            r.q_len = q_offsets[b + 1] - q_offsets[b];
            r.pos0 = start[b];
            if (r.pos0 < 0 || (int64_t)r.pos0 + r.q_len > kMaxPosition)
                return fail(KVR_ERR_OUT_OF_RANGE, "request %d: rows %d and %d more, of at most 2^24", b, r.pos0, r.q_len);
            const int64_t g0 = r.pos0 / R, g1 = r.q_len > 0 ? ((int64_t)r.pos0 + r.q_len + R - 1) / R : g0;
            r.few = INT32_MAX;
            r.off[0] = (int32_t)((int64_t)pl.ids.size() - g0);
            if ((st = take_pages(pl.ids, table, width, b, g0, g1, pages->n_pages, "page")) != KVR_OK)
                return st;
            pl.rq.push_back(r);
        }
        if ((st = check_distinct(pl.ids, 0)) != KVR_OK)
            return st;
        if (T == 0)
            return KVR_OK;
        if (!k || !v || !aligned16(k) || !aligned16(v))
            return fail(KVR_ERR_INVALID_ARG, "k / v NULL or not 16-byte aligned");
        const int64_t count[3] = {L, T, H};
        const int64_t st3[3] = {stride ? stride[0] : (int64_t)T * H * D, stride ? stride[1] : (int64_t)H * D, stride ? stride[2] : D};
        int64_t extent = D;
        for (int i = 0; i < 3; ++i) {
            if (st3[i] < 0 || st3[i] % p->vec_elems() || st3[i] > (int64_t(1) << 58) / count[i])
                return fail(KVR_ERR_INVALID_ARG, "stride[%d] = %lld must be >= 0, a multiple of %d and within 2^58 elements", i,
                            (long long)st3[i], p->vec_elems());
            extent += (count[i] - 1) * st3[i];
        }
        const Range in[2] = {range_of(k, 0, extent, p->elt()), range_of(v, 0, extent, p->elt())};
        for (const Range &x : in)
            if (x.meets(pages_range(*p, *pages, false)) || x.meets(pages_range(*p, *pages, true)))
                return fail(KVR_ERR_INVALID_ARG, "the pages overlap the new keys or values");
        cudaStream_t s = static_cast<cudaStream_t>(stream);
        if ((st = page_ready(p, pl, s)) != KVR_OK)
            return st;
        DeviceGuard g(p->device);
        page_base(*p, *pages, pl);
        PageArgs &a = pl.a;
        a.total_q = T;
        a.k = k;
        a.v = v;
        a.s_layer = st3[0];
        a.s_tok = st3[1];
        a.s_head = st3[2];
        a.turned = (flags & KVR_APPEND_TURNED) ? 1 : 0;
        if ((st = page_stage(p, pl, s)) != KVR_OK)
            return st;
        p->mark(2, s);
        NvtxRange r("kvr.k_page_append");
        const cudaError_t e = launch_page_append(a, pl.tab, p->d.dtype, D, p->n_sms, s);
        p->mark(3, s);
        if (pl.slot)
            cudaEventRecord(pl.slot->done, s);
        return e == cudaSuccess ? KVR_OK : cuda_fail(e, "page append launch");
    });
}

extern "C" kvr_status kvr_page_pack(kvr_pool_t p, const kvr_pages *pages, int32_t batch, const int32_t *table, int32_t width,
                                    const kvr_packed_pages *packed, const int32_t *packed_table, int32_t packed_width,
                                    const int32_t *begin, const int32_t *end, void *stream)
{
    return page_pack(p, pages, table, packed, packed_table, batch, width, packed_width, begin, end, false, stream);
}

extern "C" kvr_status kvr_page_unpack(kvr_pool_t p, const kvr_packed_pages *packed, int32_t batch, const int32_t *packed_table,
                                      int32_t packed_width, const kvr_pages *pages, const int32_t *table, int32_t width,
                                      const int32_t *begin, const int32_t *end, void *stream)
{
    return page_pack(p, pages, table, packed, packed_table, batch, width, packed_width, begin, end, true, stream);
}

extern "C" kvr_status kvr_page_attention(kvr_pool_t p, const kvr_pages *pages, int32_t batch, const int32_t *table, int32_t width,
                                         const int32_t *kv_len, const int32_t *q_pos, const int32_t *q_offsets, const void *q,
                                         void *out, int32_t window, int32_t n_first, const kvr_packed_pages *packed,
                                         const int32_t *packed_table, int32_t packed_width, const int32_t *packed_len,
                                         float softmax_scale, void *stream)
{
    if (!p)
        return fail(KVR_ERR_INVALID_ARG, "pool is NULL");
    if (batch < 0 || width < 0 || packed_width < 0)
        return fail(KVR_ERR_INVALID_ARG, "batch %d, widths %d, %d", batch, width, packed_width);
    if (window < 0 || n_first < 0)
        return fail(KVR_ERR_INVALID_ARG, "window %d, n_first %d", window, n_first);
    NvtxRange call("kvr_page_attention");
    return guarded([&]() -> kvr_status {
        kvr_status st;
        if ((st = check_pages(*p, pages, false)) != KVR_OK || (st = check_offsets32(q_offsets, batch, "q_offsets")) != KVR_OK ||
            (packed && (st = check_packed(*p, packed, pages->page_rows)) != KVR_OK))
            return st;
        if (batch > 0 && (!kv_len || (packed && !packed_len)))
            return fail(KVR_ERR_INVALID_ARG, "kv_len / packed_len is NULL");
        if (!(softmax_scale >= 0.f) || !std::isfinite(softmax_scale))
            return fail(KVR_ERR_INVALID_ARG, "softmax_scale %g", (double)softmax_scale);
        const int L = p->d.n_layers, Hq = p->d.n_q_heads, D = p->d.head_dim, G = Hq / p->d.n_kv_heads;
        const int32_t T = q_offsets[batch], R = pages->page_rows;
        PagePlan pl;
        pl.rq.reserve(batch);
        for (int b = 0; b < batch; ++b) {
            DevPageReq r{};
            r.q_off = q_offsets[b];
            r.q_len = q_offsets[b + 1] - q_offsets[b];
            r.kv_len = kv_len[b];
            int32_t step = std::max(1, r.q_len);   // tokens that are a request to the kernels
            if (r.kv_len < 0)
                return fail(KVR_ERR_OUT_OF_RANGE, "request %d: kv_len %d", b, r.kv_len);
            r.pos0 = q_pos ? q_pos[b] : r.kv_len - r.q_len;
            if (r.pos0 < 0 || (int64_t)r.pos0 + r.q_len > kMaxPosition)
                return fail(KVR_ERR_OUT_OF_RANGE, "request %d: positions %d and %d more, of at most 2^24", b, r.pos0, r.q_len);
            if (packed) {
                r.packed_len = packed_len[b];
                if (r.packed_len < 0 || r.packed_len > r.kv_len || r.packed_len % kPackRows)
                    return fail(KVR_ERR_OUT_OF_RANGE, "request %d: packed_len %d of %d rows, in whole blocks of %d", b, r.packed_len,
                                r.kv_len, kPackRows);
            }
            if (r.q_len > 0) {
                // rows that some query of the request sees: [0, few) and [lo, hi)
                const int64_t hi = std::min<int64_t>(r.kv_len, (int64_t)r.pos0 + r.q_len);
                const int64_t lo = std::min(hi, window > 0 ? std::max<int64_t>(0, (int64_t)r.pos0 - window + 1) : 0);
                const int64_t few = std::min<int64_t>(n_first, lo), body = r.packed_len;
                auto take = [&](int64_t a0, int64_t a1, int64_t b0, int64_t b1, bool pk, int32_t &nf, int32_t (&off)[2]) -> kvr_status {
                    // pages of rows [a0, a1), then those of [b0, b1) that are not among them
                    const int64_t p0 = a0 / R, p1 = a0 < a1 ? (a1 + R - 1) / R : p0;
                    const int64_t q1 = b0 < b1 ? (b1 + R - 1) / R : 0, q0 = std::min(std::max(p1, b0 / R), std::max(p1, q1));
                    nf = (int32_t)(a0 < a1 ? p1 : 0);
                    for (int k = 0; k < 2; ++k) {
                        const int64_t g0 = k ? q0 : p0, g1 = k ? q1 : p1;
                        off[k] = (int32_t)((int64_t)pl.ids.size() - g0);
                        kvr_status s2 = pk ? take_pages(pl.ids, packed_table, packed_width, b, g0, g1, packed->n_pages, "packed")
                                           : take_pages(pl.ids, table, width, b, g0, g1, pages->n_pages, "page");
                        if (s2 != KVR_OK)
                            return s2;
                    }
                    return KVR_OK;
                };
                if ((st = take(body, few, std::max(lo, body), hi, false, r.few, r.off)) != KVR_OK ||
                    (packed && (st = take(0, std::min(few, body), lo, std::min(hi, body), true, r.pfew, r.poff)) != KVR_OK))
                    return st;
                // a few more query rows than k_page_decode takes, on packed rows: it reads these up to three
                // times, rather than k_page_attention bf16 rows restored from them (33,280 packed rows, 256
                // units: 32 query rows in two parts 755 us, 1,657 there; 48 in three 1,132, 1,661 there; 16 x
                // 1,216, 288 units, 32 rows 650 and 1,109; four parts would be 1,300 there, for 1,120)
                const int n = G <= kPageFewRows ? (r.q_len + kPageFewRows / G - 1) / (kPageFewRows / G) : INT32_MAX;
                if (n <= kPagePackedParts && (std::min(few, body) > 0 || lo < std::min(hi, body)))
                    step = (r.q_len + n - 1) / n;
            }
            for (int32_t t = 0, n = r.q_len, pos = r.pos0; t == 0 || t < n; t += step) {
                r.q_off = q_offsets[b] + t;
                r.q_len = std::min(step, n - t);
                r.pos0 = pos + t;
                pl.rq.push_back(r);
            }
        }
        if (pl.ids.size() > INT32_MAX)
            return fail(KVR_ERR_OUT_OF_RANGE, "too many pages");
        if (T == 0)
            return KVR_OK;
        if (!q || !out || !aligned16(q) || !aligned16(out))
            return fail(KVR_ERR_INVALID_ARG, "q / out NULL or not 16-byte aligned");
        const int64_t q_rows = (int64_t)L * T * Hq, row_bytes = (int64_t)D * p->elt();
        const Range ro = range_of(out, 0, q_rows, row_bytes), rq = range_of(q, 0, q_rows, row_bytes);
        if (ro.meets(pages_range(*p, *pages, false)) || ro.meets(pages_range(*p, *pages, true)) ||
            (packed && ro.meets(packed_range(*p, *packed, R))))
            return fail(KVR_ERR_INVALID_ARG, "the output overlaps the pages");
        if (ro.meets(rq) && ro.lo != rq.lo)
            return fail(KVR_ERR_INVALID_ARG, "the output overlaps the queries (it may only be the same buffer)");
        cudaStream_t s = static_cast<cudaStream_t>(stream);
        const bool tensor = attention_tc_supported(p->d.dtype, D);
        bool few = false, many = false;   // requests for the kernel of few query rows, and for that of more
        for (const DevPageReq &r : pl.rq) {
            few = few || (r.q_len > 0 && r.q_len * (int64_t)G <= kPageFewRows);
            many = many || (tensor && r.q_len * (int64_t)G > kPageFewRows);
        }
        if ((st = check_capture(*p, s, pl.inl() && !many, "the call uses library scratch (a request of more than 16 query rows, three times "
                                                          "as many on packed rows), or uploads the tables of more than 64 "
                                                          "requests (or parts of them) or 1,024 pages")) != KVR_OK ||
            (st = ensure_device(p)) != KVR_OK)
            return st;
        DeviceGuard g(p->device);
        PageTcArgs tc{};
        PageTcMaps maps{};
        CUtensorMap mq, mk, mv, mrk, mrv;
        const int LH = L * p->d.n_kv_heads;
        int lh_slice = LH;
        if (many) {
            if (!use_tensor_cores(*p))
                return fail(KVR_ERR_UNSUPPORTED, "more than 16 query rows need the tensor-core kernel (sm_103)");
            if (q_rows > (int64_t)INT32_MAX - 256)
                return fail(KVR_ERR_UNSUPPORTED, "query rows exceed the int32 TMA coordinate range");
            if ((st = page_tc_plan(p, pl, *pages, window, n_first, tc, lh_slice)) != KVR_OK)
                return st;
            // scratch: restored keys, restored values, partial results
            const int64_t rest_rows = (int64_t)lh_slice * tc.unit_tiles * 128, rest_bytes = rest_rows * D * 2;
            const int64_t part_bytes = tc.splits > 1 ? (int64_t)lh_slice * tc.unit_items * kPagePartBytes : 0;
            if (rest_rows > (int64_t)INT32_MAX - 256)
                return fail(KVR_ERR_UNSUPPORTED, "restored rows exceed the int32 TMA coordinate range");
            if ((st = p->grow_query_scratch((size_t)(q_rows * D) * 2)) != KVR_OK ||
                (st = p->grow_part_scratch((size_t)(2 * rest_bytes + part_bytes))) != KVR_OK ||
                (st = encode_rows_map(*p, p->q_rot, q_rows, 128, &mq)) != KVR_OK)
                return st;
            tc.q_rot = p->q_rot;
            tc.rest_k = p->part;
            tc.rest_v = static_cast<char *>(p->part) + rest_bytes;
            tc.part = reinterpret_cast<float *>(static_cast<char *>(p->part) + 2 * rest_bytes);
            const int64_t rows = page_extent(*p, *pages) / D;
            if ((tc.box && ((st = encode_rows_map(*p, pages->k, rows, tc.box, &mk)) != KVR_OK ||
                            (st = encode_rows_map(*p, pages->v, rows, tc.box, &mv)) != KVR_OK)) ||
                (rest_rows && ((st = encode_rows_map(*p, tc.rest_k, rest_rows, 128, &mrk)) != KVR_OK ||
                               (st = encode_rows_map(*p, tc.rest_v, rest_rows, 128, &mrv)) != KVR_OK)))
                return st;
            tc.out32 = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
            maps = {&mq, tc.box ? &mk : &mq, tc.box ? &mv : &mq, rest_rows ? &mrk : &mq, rest_rows ? &mrv : &mq};
            // the previous call's attention must be done with the scratch
            cudaError_t e;
            if (p->q_rot_used && (e = cudaStreamWaitEvent(s, p->q_rot_done, 0)) != cudaSuccess)
                return cuda_fail(e, "query scratch ordering");
        }
        page_base(*p, *pages, pl);
        PageArgs &a = pl.a;
        a.total_q = T;
        a.q = q;
        a.out = out;
        a.scale_log2 = (softmax_scale > 0.f ? softmax_scale : 1.f / std::sqrt((float)D)) * 1.4426950408889634f;
        a.window = window;
        a.n_first = n_first;
        if (packed) {
            a.g.packed = static_cast<uint8_t *>(packed->data);
            a.g.packed_page = packed_page_bytes(*p, R);
        }
        if ((st = page_stage(p, pl, s)) != KVR_OK)
            return st;
        p->mark(4, s);
        NvtxRange r("kvr.k_page_attention");
        int32_t path = tensor ? (few ? KVR_PAGE_FEW : 0) : KVR_PAGE_CUDA_CORES;
        cudaError_t e = few && tensor ? launch_page_decode(a, pl.tab, pl.rq.data(), p->n_sms, s) : cudaSuccess;
        if (e == cudaSuccess && !tensor)
            e = launch_page_simt(a, pl.tab, p->d.dtype, D, s);
        if (e == cudaSuccess && many) {
            e = launch_page_queries(a, pl.tab, p->q_rot, s);
            int slices = 0;
            for (int lh = 0; lh < LH && e == cudaSuccess; lh += lh_slice) {
                tc.lh_base = lh;
                const int n = std::min(lh_slice, LH - lh);
                tc.total = (int64_t)n * tc.unit_items;
                e = launch_page_tc(a, tc, pl.tab, maps, n, p->n_sms, s);
                ++slices;
            }
            path |= KVR_PAGE_MANY | (tc.unit_tiles > 0 ? KVR_PAGE_RESTORED : 0) | (tc.splits > 1 ? KVR_PAGE_JOINED : 0) | slices << 8;
            cudaEventRecord(p->q_rot_done, s);
            p->q_rot_used = true;
        }
        p->page_path = path;
        p->mark(5, s);
        if (pl.slot)
            cudaEventRecord(pl.slot->done, s);
        return e == cudaSuccess ? KVR_OK : cuda_fail(e, "paged attention launch");
    });
}

// ---------------------------------------------------------------------------
// status
// ---------------------------------------------------------------------------
extern "C" kvr_status kvr_check(kvr_pool_t p, void *stream)
{
    if (!p)
        return fail(KVR_ERR_INVALID_ARG, "pool is NULL");
    kvr_status st;
    if ((st = ensure_device(p)) != KVR_OK)
        return st;
    DeviceGuard g(p->device);
    cudaError_t e;
    if ((e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream))) != cudaSuccess)
        return cuda_fail(e, "stream synchronize");
    int w = 0;
    if ((e = cudaMemcpy(&w, p->err, sizeof w, cudaMemcpyDeviceToHost)) != cudaSuccess)
        return cuda_fail(e, "error word read");
    if (w == kDevOk)
        return KVR_OK;
    cudaMemset(p->err, 0, sizeof(int));
    if (w == kDevTimeout)
        return fail(KVR_ERR_TIMEOUT, "a kernel's bounded wait ran out");
    if (w == kDevBadInput)
        return fail(KVR_ERR_DEVICE_CHECK, "an attention row's softmax denominator was not finite and positive "
                                          "(NaN or infinity in the query heads or the keys it attends to)");
    return fail(KVR_ERR_DEVICE_CHECK, "a kernel flagged device-side input (code %d)", w);
}

extern "C" const char *kvr_status_string(kvr_status s)
{
    switch (s) {
    case KVR_OK: return "KVR_OK";
    case KVR_ERR_INVALID_ARG: return "KVR_ERR_INVALID_ARG";
    case KVR_ERR_OUT_OF_RANGE: return "KVR_ERR_OUT_OF_RANGE";
    case KVR_ERR_UNSUPPORTED: return "KVR_ERR_UNSUPPORTED";
    case KVR_ERR_CUDA: return "KVR_ERR_CUDA";
    case KVR_ERR_TIMEOUT: return "KVR_ERR_TIMEOUT";
    case KVR_ERR_DEVICE_CHECK: return "KVR_ERR_DEVICE_CHECK";
    }
    return "KVR_ERR_UNKNOWN";
}

extern "C" const char *kvr_last_error(void) { return g_last_error; }

extern "C" kvr_status kvr_set_timing_events(kvr_pool_t p, void *const *events)
{
    if (!p)
        return fail(KVR_ERR_INVALID_ARG, "pool is NULL");
    p->timed = events != nullptr;
    for (int i = 0; i < 6; ++i)
        p->timing[i] = events ? static_cast<cudaEvent_t>(events[i]) : nullptr;
    return KVR_OK;
}

extern "C" kvr_status kvr_selftest_wait(kvr_pool_t p, uint64_t limit_ns, void *stream)
{
    if (!p)
        return fail(KVR_ERR_INVALID_ARG, "pool is NULL");
    kvr_status st;
    if ((st = ensure_device(p)) != KVR_OK)
        return st;
    DeviceGuard g(p->device);
    const unsigned long long lim = std::min<uint64_t>(std::max<uint64_t>(limit_ns, 1000ull), 2000000000ull);
    const cudaError_t e = launch_wait_selftest(p->err, lim, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess)
        return cuda_fail(e, "self-test launch");
    return KVR_OK;
}

extern "C" int32_t kvr_attention_path(kvr_pool_t p)
{
    if (!p)
        return -2;
    if (!p->ready)
        return KVR_PATH_UNBOUND;
    return use_tensor_cores(*p) ? KVR_PATH_TCGEN05 : KVR_PATH_CUDA_CORES;
}

extern "C" int32_t kvr_shared_path(kvr_pool_t p) { return p ? p->shared_path : -2; }
extern "C" int32_t kvr_page_path(kvr_pool_t p) { return p ? p->page_path : -2; }
