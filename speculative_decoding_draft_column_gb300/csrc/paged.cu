// libspecsel: the paged key/value cache (plan of a step, store, attention of a
// chunk of new tokens) and the rules applied to logits -- argument checks,
// launches and the C ABI.

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <initializer_list>
#include <mutex>

#include "specsel.h"
#include "common.cuh"
#include "paged.cuh"
#include "attention.cuh"
#include "logits_rules.cuh"
#include "host.h"

using host::cuda_fail;
using host::fail;

namespace {

constexpr int kMaxDevices = 64;

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

struct Device {
    bool init = false;
    int sms = 0;
    EncodeTiled encode = nullptr;
    int attn_smem[5][2];   // dynamic shared memory of the attention kernels, [shape][fp16]
};

template <int D, int QT>
constexpr int shape_index() { return D == 64 ? QT - 1 : D == 128 ? QT + 1 : 4; }

// Give an attention kernel all the shared memory a CTA can have (one CTA an SM,
// so that TMEM is never contended), and check what the kernel relies on: its
// static shared memory stays below the first 1,024-byte boundary.
template <int D, int QT, bool F16>
spec_status prepare_attention(Device &d, int smem_max)
{
    using S = attn::Shape<D, QT>;
    auto kernel = attn::attention_kernel<D, QT, F16>;
    cudaFuncAttributes at;
    cudaError_t e = cudaFuncGetAttributes(&at, kernel);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncGetAttributes");
    const int dynamic = smem_max - (int)at.sharedSizeBytes;
    if (at.sharedSizeBytes > 1024 || 1024 + S::kPayload > smem_max)
        return fail(SPEC_ERR_CUDA, "attention: %d bytes of shared memory are not enough", smem_max);
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, dynamic);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
    d.attn_smem[shape_index<D, QT>()][F16] = dynamic;
    return SPEC_OK;
}

template <int D, int QT>
spec_status prepare_attention(Device &d, int smem_max)
{
    const spec_status st = prepare_attention<D, QT, false>(d, smem_max);
    return st == SPEC_OK ? prepare_attention<D, QT, true>(d, smem_max) : st;
}

std::mutex g_paged_mu;
Device g_devices[kMaxDevices];

spec_status device(Device **out)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev < 0 || dev >= kMaxDevices) return fail(SPEC_ERR_CUDA, "device ordinal %d unsupported", dev);
    Device &d = g_devices[dev];
    std::lock_guard<std::mutex> lock(g_paged_mu);
    if (!d.init) {
        e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
        e = cudaFuncSetAttribute(paged::plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)paged::plan_smem(SPEC_PAGED_MAX_LANES));
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
        e = cudaFuncSetAttribute(rules::process_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, rules::smem_bytes(true));
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
        int smem_max = 0;
        e = cudaDeviceGetAttribute(&smem_max, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
        if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
        spec_status st = prepare_attention<64, 1>(d, smem_max);
        if (st == SPEC_OK) st = prepare_attention<64, 2>(d, smem_max);
        if (st == SPEC_OK) st = prepare_attention<128, 1>(d, smem_max);
        if (st == SPEC_OK) st = prepare_attention<128, 2>(d, smem_max);
        if (st == SPEC_OK) st = prepare_attention<256, 1>(d, smem_max);
        if (st != SPEC_OK) return st;
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
        e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found);
        if (e != cudaSuccess) return cuda_fail(e, "cudaGetDriverEntryPointByVersion");
        if (!fn || found != cudaDriverEntryPointSuccess) return fail(SPEC_ERR_CUDA, "the driver has no cuTensorMapEncodeTiled");
        d.encode = reinterpret_cast<EncodeTiled>(fn);
        d.init = true;
    }
    *out = &d;
    return SPEC_OK;
}

bool misaligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// A call's buffer, for the checks of what must not overlap.
struct Range {
    const void *p;
    int64_t bytes;
    const char *name;
};
bool overlap(const Range &a, const Range &b)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && a.bytes > 0 && b.bytes > 0 && x < y + (uint64_t)b.bytes && y < x + (uint64_t)a.bytes;
}

constexpr int64_t kMaxStride = 1ll << 39;

bool bad_stride(int64_t s) { return s < 0 || s >= kMaxStride || s % 8 != 0; }

template <bool kCooperative = false, typename K, typename A>
spec_status launch(K kernel, dim3 grid, unsigned block, size_t smem, const A &a)
{
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = host::stream();
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeCooperative;
    attr[1].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = kCooperative ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
    if (e != cudaSuccess) return cuda_fail(e, "kernel launch");
    host::count_launch();
    return SPEC_OK;
}

spec_status check_cache(const spec_paged_cache *c)
{
    if (!c || !c->k || !c->v) return fail(SPEC_ERR_ARG, "cache: null pointer");
    if (c->dtype != SPEC_BF16 && c->dtype != SPEC_F16) return fail(SPEC_ERR_ARG, "cache: unknown dtype %d", c->dtype);
    if (misaligned(c->k, 16) || misaligned(c->v, 16))
        return fail(SPEC_ERR_ARG, "cache: keys and values must be 16-byte aligned");
    if (c->pages < 1 || c->pages > INT32_MAX) return fail(SPEC_ERR_ARG, "cache: pages = %lld", (long long)c->pages);
    if (c->page_size < 1) return fail(SPEC_ERR_ARG, "cache: page_size = %d < 1", c->page_size);
    if (c->heads < 1) return fail(SPEC_ERR_ARG, "cache: heads = %d < 1", c->heads);
    if (c->head_dim < 8 || c->head_dim > 256 || c->head_dim % 8 != 0)
        return fail(SPEC_ERR_ARG, "cache: head_dim = %d, need a multiple of 8 up to 256", c->head_dim);
    if ((int64_t)c->heads * c->head_dim > INT32_MAX)
        return fail(SPEC_ERR_ARG, "cache: heads * head_dim = %lld exceeds 2^31-1", (long long)c->heads * c->head_dim);
    for (int i = 0; i < 3; ++i)
        if (bad_stride(c->k_strides[i]) || bad_stride(c->v_strides[i]))
            return fail(SPEC_ERR_ARG, "cache: strides must be non-negative multiples of 8 elements below 2^39");
    return SPEC_OK;
}

spec_status check_batch(const spec_paged_batch *b)
{
    if (!b) return fail(SPEC_ERR_ARG, "batch: null pointer");
    if (b->lanes < 0 || b->lanes > SPEC_PAGED_MAX_LANES)
        return fail(SPEC_ERR_ARG, "batch: lanes = %lld outside [0, %d]", (long long)b->lanes, SPEC_PAGED_MAX_LANES);
    if (b->max_pages < 1 || b->max_pages > INT32_MAX)
        return fail(SPEC_ERR_ARG, "batch: max_pages = %lld", (long long)b->max_pages);
    if (b->page_size < 1) return fail(SPEC_ERR_ARG, "batch: page_size = %d < 1", b->page_size);
    return SPEC_OK;
}

constexpr int64_t max2(int64_t a, int64_t b) { return a > b ? a : b; }
constexpr int64_t kPartFloats = max2(attn::Shape<128, 2>::kPartFloats, attn::Shape<256, 1>::kPartFloats);

static_assert(SPEC_PAGED_WORKSPACE_ZEROED == 2 * attn::kMaxSms * sizeof(unsigned int), "the counters");

int attention_grid(const Device &d) { return d.sms < attn::kMaxSms ? d.sms : attn::kMaxSms; }

template <int D, int QT>
spec_status launch_attention(const Device &d, const attn::Args &a, int64_t chunk, bool f16)
{
    using S = attn::Shape<D, QT>;
    static_assert(S::kPartFloats <= kPartFloats, "");
    const dim3 grid((unsigned)attention_grid(d));
    const size_t smem = (size_t)d.attn_smem[shape_index<D, QT>()][f16];
    // Whether an item's parts are joined by all its CTAs (a cooperative launch) or
    // by the last part's CTA alone (an ordinary one: 2-4 us less a call in a
    // stream, 1 in a graph; 8 lanes of 8 tokens at 8,000 keys 51.8 against 55.3 us, 64 lanes of
    // 16 tokens at 3,000 keys 30.8 against 34.8, 8 lanes of a token at 2,000 keys of one head
    // 12.0 against 14.4).  The lengths are on the device, so the number of parts is
    // estimated twice: from the items that the lanes and heads make if they are
    // even, and from one lane having all the keys (the others short, or without tokens, as in
    // a padded batch), whose heads then share the GPU.  Both are bounded by the table's
    // width and the window.  Alone, a CTA joins the even case's 128 KB in 2 us.  Of 64 lanes
    // of 4 tokens, one with 60,000 keys, it takes 29.4 against 20.5 us in a stream where that lane has
    // one head (152 parts of 8 KB), 26.6 against 23.5 where it has two (76 parts); of 64 lanes
    // of 16 tokens, one with 131,072 keys of one head (152 parts of 32 KB), 66 against 24 in a graph.
    constexpr int64_t kAlone = 32 << 10, kAloneAll = 128 << 10, kAloneWorst = 1 << 20, kAloneParts = 96;
    attn::Args b = a;
    const int64_t ctas = grid.x, rows = chunk * a.group < S::kRows ? chunk * a.group : S::kRows;
    const int64_t table = a.max_pages << a.log_page, seen = a.window > 0 && a.window < table ? a.window + S::kRows / a.group + 2 : table;
    const int64_t widest = ((seen < table ? seen : table) / S::BK + 2) / S::kLeast + 2;
    const int64_t items = (int64_t)a.lanes * a.heads_kv, likely = ctas / items + 2, one = ctas / a.heads_kv + 2;
    const int64_t parts = widest < likely ? widest : likely, worst = widest < one ? widest : one, part = rows * D * 4;
    b.share_joins = part > kAlone || parts * part > kAloneAll || worst * part > kAloneWorst || worst > kAloneParts;
    if (b.share_joins)   // CTAs wait for one another's parts
        return f16 ? launch<true>(attn::attention_kernel<D, QT, true>, grid, S::kThreads, smem, b)
                   : launch<true>(attn::attention_kernel<D, QT, false>, grid, S::kThreads, smem, b);
    return f16 ? launch(attn::attention_kernel<D, QT, true>, grid, S::kThreads, smem, b)
               : launch(attn::attention_kernel<D, QT, false>, grid, S::kThreads, smem, b);
}

// The cache as TMA sees it: [page][head][block of 64][token][64], boxes of one
// page's tokens (at most a tile's) by 64 elements -- all blocks at once where
// the box has a whole tile's rows, so that its blocks land a tile apart.
spec_status page_map(const Device &d, const spec_paged_cache &c, void *base, const int64_t *strides, CUtensorMap *map)
{
    const int tile = c.head_dim == 256 ? attn::Shape<256, 1>::BK : attn::Shape<128, 1>::BK;
    const cuuint32_t rows = (cuuint32_t)(c.page_size < tile ? c.page_size : tile);
    const cuuint64_t dims[5] = {64, (cuuint64_t)c.page_size, (cuuint64_t)c.head_dim / 64, (cuuint64_t)c.heads,
                                (cuuint64_t)c.pages};
    const cuuint64_t st[4] = {(cuuint64_t)strides[1] * 2, 128, (cuuint64_t)strides[2] * 2, (cuuint64_t)strides[0] * 2};
    const cuuint32_t box[5] = {64, rows, (int)rows == tile ? (cuuint32_t)c.head_dim / 64 : 1u, 1, 1};
    const cuuint32_t one[5] = {1, 1, 1, 1, 1};
    const CUresult r = d.encode(map, c.dtype == SPEC_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                                5, base, dims, st, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(SPEC_ERR_ARG, "cache: its layout has no tensor map (driver error %d)", (int)r);
    return SPEC_OK;
}

}  // namespace

namespace host {

cudaError_t take_paged_timeouts(unsigned int *flags)
{
    cudaError_t e = cudaMemcpyFromSymbol(flags, g_wait_timeouts, sizeof *flags);
    if (e != cudaSuccess || *flags == 0) return e;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_wait_timeouts, &zero, sizeof zero);
}

}  // namespace host

extern "C" {

spec_status spec_paged_plan(const spec_paged_batch *batch, const int32_t *free_pages, int64_t num_free,
                            const int32_t *cursor)
{
    host::clear_error();
    spec_status st = check_batch(batch);
    if (st != SPEC_OK) return st;
    const spec_paged_batch &b = *batch;
    if (b.tokens < 0) return fail(SPEC_ERR_ARG, "batch: tokens = %lld < 0", (long long)b.tokens);
    if (num_free < 0 || num_free > INT32_MAX) return fail(SPEC_ERR_ARG, "num_free = %lld", (long long)num_free);
    if (!b.cu_new || !b.info ||
        (b.lanes > 0 && (!b.context_lens || !b.new_lens || !b.held || !b.block_table || !b.seq_lens || !b.held_out)) ||
        (b.tokens > 0 && (!b.positions || !b.slots)) || (num_free > 0 && !free_pages))
        return fail(SPEC_ERR_ARG, "null pointer");
    const void *words[] = {b.context_lens, b.new_lens, b.held,      b.block_table, b.cu_new,   b.seq_lens,
                           b.held_out,     b.info,     b.positions, free_pages,    cursor};
    for (const void *p : words)
        if (misaligned(p, 4)) return fail(SPEC_ERR_ARG, "misaligned pointer (int32 arrays need 4 bytes)");
    if (misaligned(b.slots, 8)) return fail(SPEC_ERR_ARG, "misaligned pointer (slots need 8 bytes)");
    // every CTA reads the inputs while others write the outputs
    const int64_t l4 = b.lanes * 4, t4 = b.tokens < INT64_MAX / 8 ? b.tokens * 4 : INT64_MAX / 2;
    const Range in[] = {{b.context_lens, l4, "context_lens"}, {b.new_lens, l4, "new_lens"}, {b.held, l4, "held"},
                        {free_pages, num_free * 4, "free_pages"}, {cursor, 4, "cursor"}};
    const Range out[] = {{b.info, 16, "info"}, {b.held_out, l4, "held_out"}, {b.seq_lens, l4, "seq_lens"},
                         {b.cu_new, l4 + 4, "cu_new"}, {b.positions, t4, "positions"}, {b.slots, 2 * t4, "slots"},
                         {b.block_table, l4 * b.max_pages, "block_table"}};
    for (const Range &o : out)
        for (const Range &i : in)
            if (overlap(o, i)) return fail(SPEC_ERR_ARG, "outputs must not alias inputs (%s and %s)", o.name, i.name);
    Device *d = nullptr;
    st = device(&d);
    if (st != SPEC_OK) return st;
    paged::PlanArgs a = {b, free_pages, num_free, cursor};
    int64_t grid = (b.tokens + paged::kPlanThreads - 1) / paged::kPlanThreads;
    const int64_t by_lanes = (b.lanes + paged::kPlanWarps - 1) / paged::kPlanWarps;
    if (grid < by_lanes) grid = by_lanes;
    if (grid < 1) grid = 1;
    if (grid > d->sms) grid = d->sms;
    return launch(paged::plan_kernel, dim3((unsigned)grid), paged::kPlanThreads, paged::plan_smem(b.lanes), a);
}

spec_status spec_paged_store(const void *k, const void *v, int64_t tokens, int64_t k_token_stride,
                             int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                             const int64_t *slots, const spec_paged_cache *cache)
{
    host::clear_error();
    spec_status st = check_cache(cache);
    if (st != SPEC_OK) return st;
    if (tokens < 0 || tokens > INT32_MAX) return fail(SPEC_ERR_ARG, "tokens = %lld", (long long)tokens);
    if (tokens == 0) return SPEC_OK;
    if (!k || !v || !slots) return fail(SPEC_ERR_ARG, "null pointer");
    if (misaligned(k, 16) || misaligned(v, 16) || misaligned(slots, 8))
        return fail(SPEC_ERR_ARG, "misaligned pointer (keys and values need 16 bytes, slots 8)");
    if (bad_stride(k_token_stride) || bad_stride(k_head_stride) || bad_stride(v_token_stride) ||
        bad_stride(v_head_stride))
        return fail(SPEC_ERR_ARG, "strides must be non-negative multiples of 8 elements below 2^39");
    Device *d = nullptr;
    st = device(&d);
    if (st != SPEC_OK) return st;
    paged::StoreArgs a = {static_cast<const uint16_t *>(k), static_cast<const uint16_t *>(v), tokens,
                          k_token_stride, k_head_stride, v_token_stride, v_head_stride, slots, *cache};
    const int64_t nv = tokens * cache->heads * (cache->head_dim / 8);
    int64_t grid = (nv + paged::kStoreThreads - 1) / paged::kStoreThreads;
    if (grid > 8 * d->sms) grid = 8 * d->sms;
    return launch(paged::store_kernel, dim3((unsigned)grid), paged::kStoreThreads, 0, a);
}

int64_t spec_paged_attention_workspace(void)
{
    host::clear_error();
    Device *d = nullptr;
    const spec_status st = device(&d);
    if (st != SPEC_OK) return st;
    return SPEC_PAGED_WORKSPACE_ZEROED + (int64_t)attention_grid(*d) * 2 * kPartFloats * 4;
}

spec_status spec_paged_attention(const void *q, int64_t tokens, int32_t heads_q, int64_t q_token_stride,
                                 int64_t q_head_stride, const spec_paged_cache *cache, const spec_paged_batch *batch,
                                 float scale, int64_t window, int64_t max_new, void *out, float *lse,
                                 void *workspace, int64_t workspace_bytes)
{
    host::clear_error();
    spec_status st = check_cache(cache);
    if (st == SPEC_OK) st = check_batch(batch);
    if (st != SPEC_OK) return st;
    const spec_paged_cache &c = *cache;
    const spec_paged_batch &b = *batch;
    if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256)
        return fail(SPEC_ERR_ARG, "head_dim = %d: attention takes 64, 128 or 256", c.head_dim);
    if (c.page_size < 8 || (c.page_size & (c.page_size - 1)) != 0)
        return fail(SPEC_ERR_ARG, "page_size = %d: attention takes powers of two from 8", c.page_size);
    if (b.page_size != c.page_size)
        return fail(SPEC_ERR_ARG, "page_size of batch (%d) and cache (%d) differ", b.page_size, c.page_size);
    if (tokens < 0 || tokens > INT32_MAX) return fail(SPEC_ERR_ARG, "tokens = %lld", (long long)tokens);
    if (heads_q < 1 || heads_q % c.heads != 0)
        return fail(SPEC_ERR_ARG, "heads_q = %d: need a positive multiple of the cache's %d heads", heads_q, c.heads);
    if ((int64_t)tokens * heads_q > INT32_MAX) return fail(SPEC_ERR_ARG, "tokens * heads_q exceeds 2^31-1");
    // the items of the step at most: row tiles of 128 rows, a partial one for each head of a lane with tokens
    const int64_t items = tokens * heads_q / 128 + (tokens < b.lanes ? tokens : b.lanes) * c.heads;
    if (items >= 1ll << (63 - attn::kItemBit))
        return fail(SPEC_ERR_ARG, "tokens, lanes and heads make up to %lld row tiles, need fewer than 2^%d", (long long)items,
                    63 - attn::kItemBit);
    if (!(scale > 0.f) || !isfinite(scale)) return fail(SPEC_ERR_ARG, "scale = %g: must be positive and finite", scale);
    if (window < 0) return fail(SPEC_ERR_ARG, "window = %lld < 0", (long long)window);
    if (max_new < 0) return fail(SPEC_ERR_ARG, "max_new = %lld < 0", (long long)max_new);
    if (bad_stride(q_token_stride) || bad_stride(q_head_stride))
        return fail(SPEC_ERR_ARG, "strides must be non-negative multiples of 8 elements below 2^39");
    if (tokens == 0 || b.lanes == 0) return SPEC_OK;
    if (!q || !out || !b.block_table || !b.cu_new || !b.seq_lens || !workspace) return fail(SPEC_ERR_ARG, "null pointer");
    if (misaligned(q, 16) || misaligned(out, 16) || misaligned(workspace, 16) || misaligned(lse, 4) ||
        misaligned(b.block_table, 4) || misaligned(b.cu_new, 4) || misaligned(b.seq_lens, 4))
        return fail(SPEC_ERR_ARG, "misaligned pointer (q, out and workspace need 16 bytes, int32 and lse 4)");
    // from q's first element to its last, whatever lies between its rows
    const __int128 span = ((__int128)(tokens - 1) * q_token_stride + (__int128)(heads_q - 1) * q_head_stride + c.head_dim) * 2;
    const Range in[] = {{q, span < INT64_MAX ? (int64_t)span : INT64_MAX, "q"}, {b.block_table, b.lanes * b.max_pages * 4, "block_table"},
                        {b.cu_new, (b.lanes + 1) * 4, "cu_new"}, {b.seq_lens, b.lanes * 4, "seq_lens"}};
    const Range o = {out, tokens * heads_q * c.head_dim * 2, "out"}, ls = {lse, tokens * heads_q * 4, "lse"};
    for (const Range &i : in)
        for (const Range *w : {&o, &ls})
            if (overlap(*w, i)) return fail(SPEC_ERR_ARG, "%s overlaps %s", w->name, i.name);
    if (overlap(o, ls)) return fail(SPEC_ERR_ARG, "out overlaps lse");
    const int64_t need = spec_paged_attention_workspace();
    if (need < 0) return (spec_status)need;
    if (workspace_bytes < need)
        return fail(SPEC_ERR_ARG, "workspace: %lld bytes, the call needs %lld", (long long)workspace_bytes,
                    (long long)need);
    if (overlap(o, {workspace, need, ""}) || overlap(ls, {workspace, need, ""}))
        return fail(SPEC_ERR_ARG, "out or lse overlaps workspace");
    Device *d = nullptr;
    st = device(&d);
    if (st != SPEC_OK) return st;
    attn::Args a;
    memset(&a, 0, sizeof a);
    st = page_map(*d, c, c.k, c.k_strides, &a.kmap);
    if (st == SPEC_OK) st = page_map(*d, c, c.v, c.v_strides, &a.vmap);
    if (st != SPEC_OK) return st;
    a.q = static_cast<const uint16_t *>(q);
    a.tokens = tokens; a.qs_t = q_token_stride; a.qs_h = q_head_stride;
    a.heads_q = heads_q; a.heads_kv = c.heads; a.group = heads_q / c.heads;
    while ((1 << a.log_page) < c.page_size) ++a.log_page;
    while ((1u << a.group_shift) < (uint32_t)a.group) ++a.group_shift;
    a.group_magic = (uint32_t)((((1ull << a.group_shift) - a.group) << 32) / a.group + 1);
    a.block_table = b.block_table; a.cu_new = b.cu_new; a.seq_lens = b.seq_lens;
    a.lanes = (int32_t)b.lanes; a.max_pages = b.max_pages;
    // (of tiles of 64 keys, the smaller; 2^31 - 2^16 unless there are 2^15 items)
    const int64_t tiles = (1ll << attn::kItemBit) / items - 2;
    a.most_keys = (int32_t)(tiles < (0x7FFF0000 >> 6) ? tiles << 6 : 0x7FFF0000);
    a.c = scale * attn::kLog2e;
    a.window = window > INT32_MAX ? 0 : window;   // past every position: none (and positions less it stay within 64 bits)
    a.out = static_cast<uint16_t *>(out); a.lse = lse;
    a.counters = static_cast<unsigned int *>(workspace);
    a.parts = reinterpret_cast<float *>(static_cast<char *>(workspace) + SPEC_PAGED_WORKSPACE_ZEROED);
    const int64_t hint = max_new < tokens ? max_new : tokens, chunk = hint > 0 ? hint : (tokens + b.lanes - 1) / b.lanes;
    const bool two = chunk * a.group > 128;   // more rows than one tile: two tiles share every K/V tile
    const bool f16 = c.dtype == SPEC_F16;
    if (c.head_dim == 256) return launch_attention<256, 1>(*d, a, chunk, f16);
    if (c.head_dim == 128) return two ? launch_attention<128, 2>(*d, a, chunk, f16) : launch_attention<128, 1>(*d, a, chunk, f16);
    return two ? launch_attention<64, 2>(*d, a, chunk, f16) : launch_attention<64, 1>(*d, a, chunk, f16);
}

spec_status spec_logits_process(const uint16_t *logits, int64_t lanes, int32_t cols, int64_t V,
                                const int32_t *history, int64_t history_stride, const int32_t *prompt_lens,
                                const int32_t *history_lens, const int32_t *drafts, const float *penalties,
                                const int32_t *bias_ids, const float *bias_vals, int64_t max_bias,
                                const int32_t *bias_lens, const uint32_t *mask, int64_t mask_count,
                                const int32_t *mask_rows, uint16_t *out)
{
    host::clear_error();
    if (lanes < 0 || lanes > 65535) return fail(SPEC_ERR_ARG, "lanes = %lld outside [0, 65535]", (long long)lanes);
    if (cols < 1 || cols > SPEC_MAX_GAMMA + 1)
        return fail(SPEC_ERR_ARG, "cols = %d outside [1, %d]", cols, SPEC_MAX_GAMMA + 1);
    if (V < 1 || V > INT32_MAX) return fail(SPEC_ERR_ARG, "V = %lld outside [1, 2^31-1]", (long long)V);
    if (history_stride < 0 || max_bias < 0 || mask_count < 0)
        return fail(SPEC_ERR_ARG, "history_stride, max_bias and mask_count must not be negative");
    if (lanes == 0) return SPEC_OK;
    if (!logits || !out) return fail(SPEC_ERR_ARG, "null pointer");
    // (a table of no entries has no address: with its lengths or rows it is a rule that changes nothing)
    if (!!prompt_lens != !!history_lens || (history_stride > 0 ? !!history != !!prompt_lens : history && !prompt_lens))
        return fail(SPEC_ERR_ARG, "history, prompt_lens and history_lens go together");
    if (max_bias > 0 ? !!bias_ids != !!bias_vals || !!bias_ids != !!bias_lens : (bias_ids || bias_vals) && !bias_lens)
        return fail(SPEC_ERR_ARG, "bias_ids, bias_vals and bias_lens go together");
    if (mask_count > 0 ? !!mask != !!mask_rows : mask && !mask_rows)
        return fail(SPEC_ERR_ARG, "mask and mask_rows go together");
    if (misaligned(logits, 2) || misaligned(out, 2)) return fail(SPEC_ERR_ARG, "misaligned pointer (logits need 2 bytes)");
    const void *words[] = {history, prompt_lens, history_lens, drafts, penalties, bias_ids, bias_vals, bias_lens, mask, mask_rows};
    for (const void *p : words)
        if (misaligned(p, 4)) return fail(SPEC_ERR_ARG, "misaligned pointer (32-bit arrays need 4 bytes)");
    const int64_t bytes = lanes * cols * V * 2;   // below 2^16 * 2^4 * 2^31 * 2
    const char *x = reinterpret_cast<const char *>(logits), *y = reinterpret_cast<const char *>(out);
    if (x != y && x < y + bytes && y < x + bytes)
        return fail(SPEC_ERR_ARG, "out overlaps logits without being them");
    Device *d = nullptr;
    spec_status st = device(&d);
    if (st != SPEC_OK) return st;
    rules::Args a = {logits, out, lanes, V, cols, history, history_stride, prompt_lens, history_lens, drafts,
                     penalties, bias_ids, bias_vals, max_bias, bias_lens, mask, mask_count, mask_rows};
    const unsigned slices = (unsigned)((V + 7 + rules::kSlice - 1) / rules::kSlice);
    return launch(rules::process_kernel, dim3(slices, (unsigned)lanes), rules::kThreads, (size_t)rules::smem_bytes(bias_ids != nullptr), a);
}

}  // extern "C"
